"""Cases of the position-rotating appends and of latent attention, in plain form.

The operators (entry points of ``include/pagedkv.h``, called through
``paged_kv_cache_attn_gb300.binding``):

* ``rope_append``: a layer's new queries and keys rotated by position, keys
  and values written to their reserved slots of a paged pool (bf16, or e4m3
  with one power-of-two scale per block and kv-head).
* ``latent_append``: the same for a pool that holds one latent vector of 512
  and one rotated position key of 64 a token.
* ``latent_decode``: the decode step over such a pool (absorbed form): every
  query head attends to the latents themselves.
* ``latent_prefill``: new tokens of each branch attend causally to all of its
  cached tokens, with per-head keys and values expanded from the latents.

With ``own`` false everything is computed with elementary torch operations in
fp32; with ``own`` true by the library.
"""

import math

import numpy as np
import torch

own = False

BLK = 16          # tokens a block
RANK = 512        # latent vector
ROPE = 64         # rotated position key of a latent pool
NOPE = 128        # expanded key without its position part; expanded value
E_MIN, E_MAX = -126, 120


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # One decode step of a small search tree's branches: latency counts.
        {"name": "rope step 64 branches", "op": "rope_append", "kv": "bf16",
         "nb": 64, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": False,
         "ctx_lo": 1, "ctx_hi": 600, "new_lo": 1, "new_hi": 1, "salt": 1},
        # Prompts entering the cache, the 70B attention shape.
        {"name": "rope prompts 4 x 4096", "op": "rope_append", "kv": "bf16",
         "nb": 4, "Hq": 64, "Hkv": 8, "d": 128, "rot": 128, "pairs": False,
         "ctx_lo": 0, "ctx_hi": 0, "new_lo": 4096, "new_hi": 4096, "salt": 2},
        # Ragged chunks onto branches that end inside a block, e4m3 pool.
        {"name": "rope e4m3 ragged chunks", "op": "rope_append", "kv": "e4m3",
         "nb": 24, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": True,
         "ctx_lo": 3, "ctx_hi": 700, "new_lo": 37, "new_hi": 701, "salt": 3},
        # One decode step into a latent cache, all heads on one GPU.
        {"name": "latent step 128 branches", "op": "latent_append", "nb": 128,
         "Hq": 128, "pairs": True, "ctx_lo": 1, "ctx_hi": 900, "new_lo": 1,
         "new_hi": 1, "salt": 4},
        # Prompts entering a latent cache, odd lengths.
        {"name": "latent prompts 5 x ~2000", "op": "latent_append", "nb": 5,
         "Hq": 16, "pairs": False, "ctx_lo": 0, "ctx_hi": 90, "new_lo": 1801,
         "new_hi": 2203, "salt": 5},
        # One request, 16 heads (the share of one GPU in eight): latency.
        {"name": "decode 1 x 1000, 16 heads", "op": "latent_decode", "roots": 0,
         "fan": 0, "prefix": 0, "nb": 1, "lo": 1000, "hi": 1000, "Hq": 16,
         "salt": 6},
        # Independent requests of mixed lengths, all 128 heads.
        {"name": "decode 64 mixed, 128 heads", "op": "latent_decode",
         "roots": 0, "fan": 0, "prefix": 0, "nb": 64, "lo": 512, "hi": 4096,
         "Hq": 128, "salt": 7},
        # A search tree: 8 roots of 2048 tokens, 64 branches each.
        {"name": "decode fanout 8 x 64", "op": "latent_decode", "roots": 8,
         "fan": 64, "prefix": 2048, "nb": 0, "lo": 128, "hi": 900, "Hq": 16,
         "salt": 8},
        # Long contexts, few heads: the cache read is all there is.
        {"name": "decode 16 x 32768, 16 heads", "op": "latent_decode",
         "roots": 0, "fan": 0, "prefix": 0, "nb": 16, "lo": 32768, "hi": 32768,
         "Hq": 16, "salt": 9},
        # One prompt.
        {"name": "prefill 1 x 2048, 16 heads", "op": "latent_prefill", "nb": 1,
         "shared": 0, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 2048, "new_hi": 2048,
         "Hq": 16, "salt": 10},
        # Branches of one tree extended by ragged chunks.
        {"name": "prefill 6 chunks on a tree", "op": "latent_prefill", "nb": 6,
         "shared": 4096, "ctx_lo": 1, "ctx_hi": 200, "new_lo": 99,
         "new_hi": 705, "Hq": 32, "salt": 11},
        # A long prompt.
        {"name": "prefill 1 x 8192, 32 heads", "op": "latent_prefill", "nb": 1,
         "shared": 0, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 8192, "new_hi": 8192,
         "Hq": 32, "salt": 12},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    salt = rng.randrange(1, 1 << 20)
    op = rng.choice(["rope_append", "latent_append", "latent_decode",
                     "latent_prefill"])
    if op in ("rope_append", "latent_append"):
        step = rng.random() < 0.4
        nb = log(1, 256) if step else log(1, 16)
        lo = 1 if step else log(2, 1500)
        hi = 1 if step else lo + rng.randrange(0, 300)
        c = {"op": op, "nb": nb, "pairs": rng.random() < 0.5,
             "ctx_lo": rng.randrange(0, 40), "ctx_hi": rng.randrange(40, 700),
             "new_lo": lo, "new_hi": hi, "salt": salt}
        if op == "latent_append":
            return {**c, "Hq": rng.choice([1, 8, 16, 32, 128])}
        hkv = rng.choice([1, 2, 8])
        d = rng.choice([64, 128])
        return {**c, "kv": rng.choice(["bf16", "e4m3"]), "Hkv": hkv,
                "Hq": hkv * rng.choice([1, 4, 8]), "d": d,
                "rot": rng.choice([d, d // 2])}
    if op == "latent_decode":
        hq = rng.choice([4, 16, 32, 128])
        if rng.random() < 0.5:
            lo = log(1, 4000)
            return {"op": op, "roots": 0, "fan": 0, "prefix": 0,
                    "nb": log(1, 64), "lo": lo, "hi": lo + rng.randrange(0, 900),
                    "Hq": hq, "salt": salt}
        return {"op": op, "roots": rng.randrange(1, 5),
                "fan": rng.randrange(2, 33), "prefix": 16 * rng.randrange(1, 128),
                "nb": 0, "lo": rng.randrange(1, 60),
                "hi": rng.randrange(60, 600), "Hq": hq, "salt": salt}
    nb = rng.randrange(1, 6)
    lo = log(1, 1200)
    return {"op": op, "nb": nb, "shared": rng.choice([0, 16 * rng.randrange(1, 64)]),
            "ctx_lo": 0, "ctx_hi": rng.randrange(1, 300), "new_lo": lo,
            "new_hi": lo + rng.randrange(0, 300), "Hq": rng.choice([2, 8, 16, 32]),
            "salt": salt}


# ---- lengths: a function of the case alone -----------------------------------

def _u(case, what, lo, hi, n):
    g = np.random.default_rng([case["salt"], what])
    return g.integers(lo, hi, size=n, endpoint=True).astype(np.int64)


def _lens(case):
    """(context before the call, new tokens) of every branch; for decode (all
    cached tokens, 1)."""
    if case["op"] == "latent_decode":
        n = case["roots"] * case["fan"] if case["roots"] else case["nb"]
        own_len = _u(case, 0, case["lo"], case["hi"], n)
        return own_len + case["prefix"], np.ones(n, np.int64)
    nb = case["nb"]
    ctx = _u(case, 0, case["ctx_lo"], case["ctx_hi"], nb) + case.get("shared", 0)
    return ctx, _u(case, 1, case["new_lo"], case["new_hi"], nb)


def _layout(case, total_lens):
    """(block tables [nb][max_blocks], segments, blocks of the pool): shared
    prefixes once, everything else apart, in a random physical order."""
    nb = len(total_lens)
    nblk = -(-total_lens // BLK)
    if case["op"] == "latent_decode" and case["roots"]:
        run, pre = case["fan"], case["prefix"] // BLK
    else:
        run, pre = nb, case.get("shared", 0) // BLK
    if nb == 1:
        pre = 0
    n_runs = nb // run if pre else 0
    blocks = int((nblk - pre).sum()) + n_runs * pre
    order = np.random.default_rng([case["salt"], 7]).permutation(blocks)
    tables = np.full((nb, int(nblk.max())), -1, np.int32)
    groups, at = [], 0
    for r in range(n_runs):
        tables[r * run:(r + 1) * run, :pre] = order[at:at + pre]
        groups.append((r * run, run, 0, pre))
        at += pre
    for b in range(nb):
        k = int(nblk[b]) - pre
        tables[b, pre:pre + k] = order[at:at + k]
        at += k
    return tables, np.asarray(groups, np.int32).reshape(-1, 4), blocks


def work(case):
    ctx, new = _lens(case)
    n = int(new.sum())
    op = case["op"]
    if op == "rope_append":
        hq, hkv, d = case["Hq"], case["Hkv"], case["d"]
        e = 1 if case["kv"] == "e4m3" else 2
        by = n * (4 * hq * d + 4 * hkv * d + 4 * case["rot"] + 2 * e * hkv * d)
        return {"bytes": by, "flops": n * (hq + hkv) * case["rot"] * 3}
    if op == "latent_append":
        by = n * (2 * 2 * (RANK + ROPE) + 4 * case["Hq"] * ROPE + 4 * ROPE)
        return {"bytes": by, "flops": n * (case["Hq"] + 1) * ROPE * 3}
    hq = case["Hq"]
    if op == "latent_decode":
        uniq = int(ctx.sum())
        if case["roots"]:
            uniq -= case["roots"] * (case["fan"] - 1) * case["prefix"]
        nb = len(ctx)
        return {"bytes": uniq * 2 * (RANK + ROPE) + nb * hq * 2 * (2 * RANK + ROPE),
                "flops": 2 * (2 * RANK + ROPE) * hq * int(ctx.sum())}
    total = ctx + new
    uniq = int(total.sum()) - (case["nb"] - 1) * case["shared"]
    pairs = int((new * ctx + new * (new + 1) // 2).sum())
    return {"bytes": uniq * 2 * (RANK + ROPE) + 4 * hq * NOPE * RANK +
            n * hq * 2 * (2 * NOPE + ROPE),
            "flops": 2 * RANK * 2 * NOPE * hq * uniq +
            2 * (2 * NOPE + ROPE) * hq * pairs}


# ---- inputs ------------------------------------------------------------------

def _rope_table(n, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    ang = np.arange(max(n, 1))[:, None] * inv[None, :]
    t = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    return torch.from_numpy(t).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["salt"])

    def rn(*shape, gain=1.0, dtype=torch.bfloat16):
        # In pieces of one dtype, so that a large pool needs no fp32 copy.
        x = torch.empty(shape, dtype=dtype, device="cuda")
        x.normal_(0.0, gain, generator=g)
        return x

    op = case["op"]
    ctx, new = _lens(case)
    total = ctx if op == "latent_decode" else ctx + new
    tables, groups, blocks = _layout(case, total)
    nb, n = len(total), int(new.sum())
    s = {"case": case, "nb": nb, "n": n, "blocks": blocks,
         "mb": tables.shape[1], "hgroups": groups, "htables": tables,
         "hlens": total.astype(np.int32), "hnew": new.astype(np.int32),
         "tables": torch.from_numpy(tables).cuda(),
         "lens": torch.from_numpy(total.astype(np.int32)).cuda(),
         "groups": torch.from_numpy(groups.copy() if len(groups) else
                                    np.zeros((1, 4), np.int32)).cuda(),
         "status": torch.zeros(256, dtype=torch.uint8, device="cuda")}
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["hoff"] = off
    s["off"] = torch.from_numpy(off).cuda()
    # A step of one new token a branch needs no offsets.
    s["off_arg"] = None if (new == 1).all() else s["off"]
    if op in ("rope_append", "latent_append"):
        rot = case["rot"] if op == "rope_append" else ROPE
        s["rope"] = _rope_table(int(total.max()), rot)
    if op == "rope_append":
        hq, hkv, d = case["Hq"], case["Hkv"], case["d"]
        # One fused projection's rows: q, k and v are slices of it.
        qkv = rn(n, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(n, hkv, d)
        s["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        if case["kv"] == "bf16":
            s["k_pool"] = rn(blocks, hkv, BLK, d)
            s["v_pool"] = rn(blocks, hkv, BLK, d)
            s["scales"] = None
        else:
            s["k_pool"], s["v_pool"] = (
                torch.randint(0, 255, (blocks, hkv, BLK * d), generator=g,
                              dtype=torch.uint8, device="cuda") for _ in "kv")
            for p in (s["k_pool"], s["v_pool"]):
                p[(p & 127) == 127] = 0            # no NaN codes
            s["scales"] = torch.zeros(blocks, hkv, 4, device="cuda")
            e = torch.randint(-9, -5, (blocks, hkv, 2), generator=g,
                              device="cuda")
            s["scales"][..., :2] = torch.exp2(e.float())
        return s
    s["c_pool"] = rn(blocks, BLK, RANK)
    s["r_pool"] = rn(blocks, BLK, ROPE)
    hq = case["Hq"]
    if op == "latent_append":
        # The down-projection's row: latent and position key side by side; the
        # position part of q is a slice of its projection, and goes into the
        # absorbed query's row.
        row = rn(n, RANK + ROPE)
        s["c"], s["r"] = row[:, :RANK], row[:, RANK:]
        s["q"] = rn(n, hq, NOPE + ROPE)[:, :, NOPE:]
        s["q_row"] = torch.zeros(n, hq, RANK + ROPE, dtype=torch.bfloat16,
                                 device="cuda")
        return s
    s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
    if op == "latent_decode":
        # An absorbed query: its products with latents of unit variance have
        # the spread that unit queries have with unit keys.
        s["q"] = torch.cat([rn(nb, hq, RANK, gain=0.5), rn(nb, hq, ROPE)], -1)
        s["out"] = torch.zeros(nb, hq, RANK, dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = rn(n, hq, NOPE + ROPE)
        s["w"] = rn(hq, 2 * NOPE, RANK, gain=1.0 / math.sqrt(RANK))
        s["out"] = torch.zeros(n, hq, NOPE, dtype=torch.bfloat16, device="cuda")
    if own:
        from paged_kv_cache_attn_gb300 import binding as B
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        if op == "latent_decode":
            plan, s["info"] = B.paged_decode_plan(
                nb, hq, 1, RANK, s["mb"], s["hlens"], groups, sms,
                B.KV_PLAN_LATENT)
        else:
            plan, s["info"] = B.paged_latent_prefill_plan(
                nb, hq, blocks, tables, s["hlens"], s["hnew"], sms)
        s["plan"] = torch.from_numpy(plan).cuda()
        s["ws"] = torch.empty(s["info"].workspace_bytes, dtype=torch.uint8,
                              device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _tokens(s):
    """(branch, position, physical block, slot) of every new token."""
    cnt = s["off"][1:] - s["off"][:-1]
    b = torch.repeat_interleave(torch.arange(s["nb"], device="cuda"), cnt.long(),
                                output_size=s["n"])
    i = torch.arange(s["n"], device="cuda") - s["off"][b]
    pos = (s["lens"][b] - cnt[b]) + i
    return b, pos.long(), s["tables"][b, pos // BLK].long(), (pos % BLK).long()


def _rotate(x, table, pos, pairs):
    """x [n][heads][d] in fp32: its first table.shape[1] * 2 dimensions rotated."""
    h = table.shape[1]
    cs = table[pos][:, None]
    c, si = cs[..., 0], cs[..., 1]
    x = x.float()
    if pairs:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack([a * c - b * si, b * c + a * si], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat([a * c - b * si, b * c + a * si], -1)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _exponent(amax):
    """Smallest e in range with amax <= 448 * 2^e."""
    m, k = torch.frexp(amax)                 # amax = m 2^k, m in [0.5, 1)
    e = torch.where(m <= 0.875, k - 9, k - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e in fp32, exactly (0 below the normal range)."""
    e = e.int()
    return torch.where(e < E_MIN, 0, (e + 127) << 23).view(torch.float32)


def _tile_offsets(d, transposed):
    t = torch.arange(BLK, device="cuda")[:, None]
    c = torch.arange(d, device="cuda")[None, :]
    if transposed:
        return c * BLK + t
    return t * d + ((((c >> 4) ^ (t & 7)) << 4) + (c & 15) if d == 128 else c)


def _write_e4m3(pool, scale, x, phys, slot, transposed):
    """x [n][Hkv][d] fp32 into slots of pool [blocks][Hkv][16 d], scale
    [blocks][Hkv], under the block rule."""
    n, hkv, d = x.shape
    blk, g = torch.unique(phys, return_inverse=True)
    rows = torch.full((len(blk), BLK), -1, dtype=torch.long, device="cuda")
    rows[g, slot] = torch.arange(n, device="cuda")
    put = rows >= 0
    xt = torch.where(put[:, :, None, None], x[rows.clamp(min=0)], 0.0)
    xt = xt.permute(0, 2, 1, 3)                                # [G][Hkv][16][d]
    e_new = _exponent(xt.abs().amax((2, 3)))
    e_old = torch.frexp(scale[blk])[1] - 1
    e = torch.where(put[:, :1], e_new, torch.maximum(e_old, e_new))
    off = _tile_offsets(d, transposed).reshape(-1)
    codes = pool[blk][:, :, off].view(len(blk), hkv, BLK, d)
    old = codes.view(torch.float8_e4m3fn).float()
    old = (old * _pow2(e_old - e)[:, :, None, None]).to(torch.float8_e4m3fn)
    enc = (xt * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn)
    first = torch.where(put, torch.arange(BLK, device="cuda"), BLK).amin(1)
    before = torch.arange(BLK, device="cuda")[None] < first[:, None]
    res = torch.where(put[:, None, :, None], enc.view(torch.uint8),
                      torch.where(before[:, None, :, None],
                                  old.view(torch.uint8), codes))
    tile = torch.empty_like(pool[blk])
    tile[:, :, off] = res.reshape(len(blk), hkv, -1)
    pool[blk] = tile
    scale[blk] = _pow2(e)


def _plain_rope_append(s):
    case = s["case"]
    b, pos, phys, slot = _tokens(s)
    k = _rotate(s["k"], s["rope"], pos, case["pairs"])
    s["q_out"].copy_(_rotate(s["q"], s["rope"], pos, case["pairs"]))
    if case["kv"] == "bf16":
        s["k_pool"][phys, :, slot] = k.bfloat16()
        s["v_pool"][phys, :, slot] = s["v"]
        return s["q_out"], s["k_pool"], s["v_pool"]
    _write_e4m3(s["k_pool"], s["scales"][..., 0], k, phys, slot, False)
    _write_e4m3(s["v_pool"], s["scales"][..., 1], s["v"].float(), phys, slot, True)
    return _e4m3_outputs(s)


def _e4m3_outputs(s):
    return (s["q_out"], s["k_pool"].view(torch.float8_e4m3fn),
            s["v_pool"].view(torch.float8_e4m3fn), s["scales"])


def _plain_latent_append(s):
    b, pos, phys, slot = _tokens(s)
    pairs = s["case"]["pairs"]
    s["c_pool"][phys, slot] = s["c"]
    s["r_pool"][phys, slot] = _rotate(s["r"][:, None], s["rope"], pos,
                                      pairs)[:, 0].bfloat16()
    s["q_row"][..., RANK:] = _rotate(s["q"], s["rope"], pos, pairs).bfloat16()
    return s["q_row"], s["c_pool"], s["r_pool"]


def _cached(s):
    t = s["tables"].clamp(min=0).long()
    c = s["c_pool"][t].flatten(1, 2).float()                  # [nb][L][512]
    return c, s["r_pool"][t].flatten(1, 2).float()


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_latent_decode(s):
    c, r = _cached(s)
    q = s["q"].float() * s["scale"]
    x = q[..., :RANK] @ c.transpose(1, 2) + q[..., RANK:] @ r.transpose(1, 2)
    seen = torch.arange(c.shape[1], device="cuda") < s["lens"][:, None]
    p = _softmax(torch.where(seen[:, None], x, -math.inf))
    s["out"].copy_(p @ c)
    return s["out"]


def _plain_latent_prefill(s):
    c, r = _cached(s)
    hq, nb, n = s["case"]["Hq"], s["nb"], s["n"]
    kv = c[:, None] @ s["w"].float().transpose(1, 2)          # [nb][Hq][L][256]
    b, pos, _, _ = _tokens(s)
    i = torch.arange(n, device="cuda") - s["off"][b]
    m = int(s["hnew"].max())
    q = torch.zeros(nb, m, hq, NOPE + ROPE, device="cuda")
    q[b, i] = s["q"].float() * s["scale"]
    at = torch.zeros(nb, m, dtype=torch.long, device="cuda")
    at[b, i] = pos
    q = q.transpose(1, 2)                                     # [nb][Hq][m][192]
    x = q[..., :NOPE] @ kv[..., :NOPE].transpose(2, 3)
    x += q[..., NOPE:] @ r[:, None].transpose(2, 3)
    seen = torch.arange(c.shape[1], device="cuda") <= at[:, :, None]
    x.masked_fill_(~seen[:, None], -math.inf)
    y = _softmax(x) @ kv[..., NOPE:]
    s["out"].copy_(y.transpose(1, 2)[b, i])
    return s["out"]


_run_plain = {"rope_append": _plain_rope_append,
              "latent_append": _plain_latent_append,
              "latent_decode": _plain_latent_decode,
              "latent_prefill": _plain_latent_prefill}


# ---- the library's calls -----------------------------------------------------

def _own_rope_append(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    style = B.KV_ROPE_PAIRS if c["pairs"] else B.KV_ROPE_HALVES
    if c["kv"] == "bf16":
        B.paged_rope_append(
            s["q"], s["k"], s["v"], s["rope"], style, s["q_out"], s["k_pool"],
            s["v_pool"], s["blocks"], s["tables"], s["lens"], s["off_arg"],
            s["n"], s["nb"], s["mb"], c["Hq"], c["Hkv"], c["d"], s["status"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    B.paged_rope_append_e4m3(
        s["q"], s["k"], s["v"], s["rope"], style, s["q_out"], s["k_pool"],
        s["v_pool"], s["scales"], s["blocks"], s["tables"], s["lens"],
        s["off_arg"], s["n"], s["nb"], s["mb"], c["Hq"], c["Hkv"], c["d"],
        s["status"])
    return _e4m3_outputs(s)


def _own_latent_append(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    style = B.KV_ROPE_PAIRS if c["pairs"] else B.KV_ROPE_HALVES
    B.paged_latent_append(
        s["c"], s["r"], s["q"], s["rope"], style, s["q_row"][..., RANK:],
        s["c_pool"], s["r_pool"], s["blocks"], s["tables"], s["lens"],
        s["off_arg"], s["n"], s["nb"], s["mb"], c["Hq"], s["status"])
    return s["q_row"], s["c_pool"], s["r_pool"]


def _own_latent_decode(s):
    from paged_kv_cache_attn_gb300 import binding as B
    B.paged_latent_decode_attn(
        s["q"], s["c_pool"], s["r_pool"], s["blocks"], s["tables"], s["lens"],
        s["groups"], len(s["hgroups"]), s["nb"], s["mb"], s["case"]["Hq"],
        s["scale"], s["out"], s["plan"], s["info"], s["ws"], s["ws"].numel())
    return s["out"]


def _own_latent_prefill(s):
    from paged_kv_cache_attn_gb300 import binding as B
    B.paged_latent_prefill_attn(
        s["q"], s["c_pool"], s["r_pool"], s["blocks"], s["w"], s["n"],
        s["nb"], s["case"]["Hq"], s["scale"], s["out"], s["plan"], s["info"],
        s["ws"], s["ws"].numel())
    return s["out"]


_run_own = {"rope_append": _own_rope_append,
            "latent_append": _own_latent_append,
            "latent_decode": _own_latent_decode,
            "latent_prefill": _own_latent_prefill}


# ---- the definition in 64 bits -----------------------------------------------

def _exact_rotation(x, p, rot, pairs, table):
    """One token's heads [heads][d] in float64, as complex numbers times
    c + i s (the table's values, taken as they are)."""
    x = x.double()
    w = torch.complex(table[p, :, 0].double(), table[p, :, 1].double())
    y = x.clone()
    if pairs:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * w[:, None]
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        h = rot // 2
        z = torch.complex(x[..., :h], x[..., h:rot]) * w[:, None]
        y[..., :h], y[..., h:rot] = z.real, z.imag
    return y


def _exact_pow2(e):
    """2^e in float64 from its bits (exp2 need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_log2(x):
    """floor(log2 x) of positive normal float64 values, from their bits."""
    return (x.contiguous().view(torch.int64) >> 52) - 1023


def _exact_e4m3(x):
    """Nearest e4m3 value, ties to even, |x| <= 448."""
    lg = _exact_log2(x.abs().clamp(min=2.0 ** -20))
    step = _exact_pow2(lg.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    off, lens, tab = s["hoff"], s["hlens"], s["htables"]
    if op in ("rope_append", "latent_append"):
        pos = np.concatenate([np.arange(lens[b] - (off[b + 1] - off[b]), lens[b])
                              for b in range(s["nb"])])
        brn = np.repeat(np.arange(s["nb"]), off[1:] - off[:-1])
        phys = torch.from_numpy(tab[brn, pos // BLK].astype(np.int64)).cuda()
        slot = torch.from_numpy(pos % BLK).cuda()
        p = torch.from_numpy(pos).cuda()
        pairs = case["pairs"]
        rot = case["rot"] if op == "rope_append" else ROPE
        q = _exact_rotation(s["q"], p, rot, pairs, s["rope"])
        if op == "latent_append":
            row = s["q_row"].double()
            row[..., RANK:] = q
            c, r = s["c_pool"].double(), s["r_pool"].double()
            c[phys, slot] = s["c"].double()
            r[phys, slot] = _exact_rotation(s["r"][:, None], p, rot, pairs,
                                            s["rope"])[:, 0]
            return row, c, r
        k = _exact_rotation(s["k"], p, rot, pairs, s["rope"])
        v = s["v"].double()
        if case["kv"] == "bf16":
            kp, vp = s["k_pool"].double(), s["v_pool"].double()
            kp[phys, :, slot] = k
            vp[phys, :, slot] = v
            return q, kp, vp
        if s["n"] > 20000:
            return None
        d, outs = case["d"], [q]
        sc = s["scales"].double()
        where = {}
        for t in range(s["n"]):
            where.setdefault((int(brn[t]), int(pos[t]) // BLK), []).append(t)
        for x, pool, col in ((k, s["k_pool"], 0), (v, s["v_pool"], 1)):
            val = pool.view(torch.float8_e4m3fn).double()
            o = _tile_offsets(d, col == 1)
            for (b, lb), ts in where.items():
                blk, s0 = int(tab[b, lb]), int(pos[ts[0]]) % BLK
                rows = x[ts[0]:ts[-1] + 1]                    # [m][Hkv][d]
                amax = rows.abs().amax((0, 2))
                e = _exact_log2(amax.clamp(min=2.0 ** -200)) - 9
                e = (e + (amax > 448.0 * _exact_pow2(e)).long())
                e = (e + (amax > 448.0 * _exact_pow2(e)).long()).clamp(E_MIN, E_MAX)
                if s0:
                    e0 = _exact_log2(sc[blk, :, col])
                    e = torch.maximum(e, e0)
                    old = val[blk][:, o[:s0].reshape(-1)]
                    val[blk, :, o[:s0].reshape(-1)] = _exact_e4m3(
                        old * _exact_pow2(e0 - e)[:, None])
                sc[blk, :, col] = _exact_pow2(e)
                y = _exact_e4m3(rows * _exact_pow2(-e)[None, :, None])
                val[blk, :, o[s0:s0 + len(ts)].reshape(-1)] = \
                    y.transpose(0, 1).flatten(1)
            outs.append(val)
        return (*outs, sc)
    hq = case["Hq"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(s["nb"]):
        L = int(lens[b])
        ids = torch.from_numpy(tab[b, :-(-L // BLK)].astype(np.int64)).cuda()
        c = s["c_pool"][ids].reshape(-1, RANK)[:L].double()
        r = s["r_pool"][ids].reshape(-1, ROPE)[:L].double()
        if op == "latent_decode":
            x = s["q"][b].double() @ torch.cat([c, r], 1).T * s["scale"]
            out[b] = torch.softmax(x, -1) @ c
            continue
        m = int(off[b + 1] - off[b])
        see = torch.ones(m, L, dtype=torch.bool, device="cuda").tril(L - m)
        for h in range(hq):
            k = torch.cat([c @ s["w"][h, :NOPE].double().T, r], 1)
            x = s["q"][off[b]:off[b + 1], h].double() @ k.T * s["scale"]
            x[~see] = -math.inf
            out[off[b]:off[b + 1], h] = torch.softmax(x, -1) @ (
                c @ s["w"][h, NOPE:].double().T)
    return out
