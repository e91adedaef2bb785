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
