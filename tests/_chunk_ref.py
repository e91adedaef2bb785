"""Attention over a GQA pool in 64 bits, written from its formula, and inputs for
its tests (torch on any device)."""

import torch

BLK = 16


def pool(blocks, Hkv, d, g, kv="bf16", device="cuda"):
    """(k_pool, v_pool, scales, keys, values): a pool of unit values, and what it
    holds as float64 [blocks][Hkv][16][d]."""
    if kv == "bf16":
        k, v = (torch.randn(blocks, Hkv, BLK, d, generator=g, device=device)
                .bfloat16() for _ in "kv")
        return k, v, None, k.double(), v.double()
    out, vals = [], []
    scales = torch.zeros(blocks, Hkv, 4, device=device)
    for i in range(2):
        x = torch.randn(blocks, Hkv, BLK, d, generator=g, device=device)
        e = torch.randint(-9, -6, (blocks, Hkv), generator=g, device=device)
        s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        code = (x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        vals.append(code.double() * s.double()[..., None, None])
        t = torch.arange(BLK, device=device)[:, None]
        c = torch.arange(d, device=device)[None]
        if i == 1:
            at = c * BLK + t
        elif d == 128:
            at = t * d + (((c >> 4) ^ (t & 7)) << 4) + (c & 15)
        else:
            at = t * d + c
        tile = torch.zeros(blocks, Hkv, BLK * d, dtype=torch.uint8, device=device)
        tile[:, :, at.reshape(-1)] = code.view(torch.uint8).flatten(2)
        out.append(tile)
        scales[..., i] = s
    return out[0], out[1], scales, vals[0], vals[1]


def rows(x, table, L, h):
    """[L][d] of kv-head h of a branch from float64 [blocks][Hkv][16][d]."""
    t = torch.as_tensor(table[:-(-L // BLK)], dtype=torch.long, device=x.device)
    return x[t, h].reshape(-1, x.shape[-1])[:L]


def attend(q, k, v, scale, pos):
    """q [n][d], k, v [L][d], pos [n]: (out [n][d], bound on its error).

    Bound: the weights are rounded to bf16 (half a step, 2^-8 of each); a score is
    a sum of d products in fp32 (d x 2^-23 of the products' magnitudes), times the
    scale (2^-23), and moves a weight by exp(+-delta), the normalisation by the
    weighted mean of those; the sum over L tokens adds L x 2^-23 and the
    exponential and the joins less than 2^-18, relative to sum_t w_t |v_t|; the
    result is rounded to bf16 once (2^-8)."""
    q = q.double()
    s = q @ k.T * scale
    see = torch.arange(k.shape[0], device=q.device)[None] <= pos[:, None]
    s = s.masked_fill(~see, float("-inf"))
    p = torch.softmax(s, -1)
    out = p @ v
    ds = (q.abs() @ k.abs().T) * scale * (q.shape[1] + 1) * 2.0 ** -23
    ds = ds.masked_fill(~see, 0.0)
    mean = (p * ds).sum(-1, keepdim=True)
    rel = 2.0 ** -8 + k.shape[0] * 2.0 ** -23 + 2.0 ** -18
    err = (p * torch.expm1(ds + mean)) @ v.abs() + (p @ v.abs()) * rel
    return out, err * (1 + 2.0 ** -6) + out.abs() * 2.0 ** -8
