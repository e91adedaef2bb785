"""Latent attention in 64 bits (torch on the GPU), written from its formulas."""

import torch


def tokens(pool, table, L):
    """[L][width] rows of one layer's pool [blocks][1][16][width]."""
    t = torch.as_tensor(table[:-(-L // 16)], dtype=torch.long, device=pool.device)
    return pool[t].reshape(-1, pool.shape[-1])[:L].double()


def decode(q, c, r, scale):
    """q [rows][576], c [L][512], r [L][64]: (out, bound on its error).

    Bound: the weights are rounded to bf16 (half a step, 2^-8 of each), the
    scores are sums of 576 products in fp32 (576 x 2^-23 of the products'
    magnitudes, twice that on a weight), the sum over L tokens adds L x 2^-23
    and the exponential and the merges less than 2^-18, all relative to
    sum_t w_t |c_t|; the result is rounded to bf16 once."""
    q = q.double()
    k = torch.cat([c, r], 1)
    s = q @ k.T * scale
    w = torch.softmax(s, -1)
    out = w @ c
    mag = w @ c.abs()
    ds = (q.abs() @ k.abs().T * scale).amax(-1, keepdim=True) * 576 * 2.0 ** -23
    rel = 2.0 ** -8 + 2 * ds + c.shape[0] * 2.0 ** -23 + 2.0 ** -18
    return out, mag * rel + out.abs() * 2.0 ** -8


def prefill(q, c, r, w, scale, pos):
    """One branch and head: q [n][192], c [L][512], r [L][64], w [256][512],
    pos [n]: (out [n][128], bound on its error).

    Bound: keys and values are sums of 512 products in fp32 (512 x 2^-23 of the
    products' magnitudes) rounded to bf16 (2^-8); weights are rounded to bf16
    (2^-8); a score is a sum of 192 products in fp32 of the rounded keys; the
    sum over tokens and the exponential as for decode; the result is rounded
    once (2^-8).  A score's error delta moves a weight by the factor
    exp(+-delta), and the normalisation by no more."""
    q, w = q.double(), w.double()
    k0, v = c @ w[:128].T, c @ w[128:].T
    acc = 512 * 2.0 ** -23
    dk = k0.abs() * 2.0 ** -8 + (c.abs() @ w[:128].abs().T) * acc
    dv = v.abs() * 2.0 ** -8 + (c.abs() @ w[128:].abs().T) * acc
    k = torch.cat([k0, r], 1)
    s = q @ k.T * scale
    see = torch.arange(k.shape[0], device=q.device)[None] <= pos[:, None]
    s = s.masked_fill(~see, float("-inf"))
    p = torch.softmax(s, -1)
    out = p @ v
    ds = (q[:, :128].abs() @ dk.T + (q.abs() @ k.abs().T) * 192 * 2.0 ** -23) \
        * scale
    ds = ds.masked_fill(~see, 0.0)
    # Weighted, not the worst: each weight carries its own score's error, and
    # the normalisation their weighted mean.
    mean = (p * ds).sum(-1, keepdim=True)
    rel = 2.0 ** -8 + k.shape[0] * 2.0 ** -23 + 2.0 ** -18
    err = (p * torch.expm1(ds + mean)) @ v.abs() + p @ dv + (p @ v.abs()) * rel
    return out, err * (1 + 2.0 ** -6) + out.abs() * 2.0 ** -8
