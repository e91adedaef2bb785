"""Position rotation in 64 bits, written from its definition."""

import numpy as np
import torch


def table(n, rot, base=10000.0):
    """fp32 (cos, sin) of every position: [n][rot / 2][2]."""
    inv = base ** (-np.arange(rot // 2) * 2.0 / rot)
    ang = np.arange(n)[:, None] * inv[None, :]
    return torch.from_numpy(
        np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32))


def rotate(x, tab, pos, pairs):
    """x [n][heads][d], pos [n]: (rotated in float64, sum of the two products'
    magnitudes, for error bounds)."""
    x = x.double()
    h = tab.shape[1]
    t = tab.to(x.device)[pos].double()
    c, s = t[:, None, :, 0], t[:, None, :, 1]
    ia = torch.arange(h, device=x.device) * (2 if pairs else 1)
    ib = ia + (1 if pairs else h)
    a, b = x[..., ia], x[..., ib]
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def bf16_bound(y, mag):
    """One rounding to bf16 (half a step: 2^-8 relative) after two fp32
    roundings of the products and their sum (2^-24 of each, counted twice)."""
    return y.abs() * 2.0 ** -8 + mag * 2.0 ** -22


def positions(lens, counts):
    """(branch, position) of every new token, from host lists."""
    b = np.repeat(np.arange(len(lens)), counts)
    p = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, counts)]) \
        if len(lens) else np.zeros(0)
    return b.astype(np.int64), p.astype(np.int64)
