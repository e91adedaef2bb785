"""Cases of chunk attention, of decode steps over selected blocks and of beam
selection, in plain form.

The operators (entry points of ``include/pagedkv.h``, called through
``paged_kv_cache_attn_gb300.binding``):

* ``chunk``: new tokens of each branch (a prompt, a chunk of one, drafted tokens,
  one token) attend causally to all cached tokens of their branch in a paged pool
  (bf16, or e4m3 with one power-of-two scale per block and kv-head).
* ``bounds``: per block and kv-head, the least and the largest value of every key
  dimension as whole numbers of 8 bits times a power of two, brought up to date
  for the blocks that hold new tokens.
* ``sparse``: a decode step over the blocks whose bounds promise the highest
  scores: selection per branch and kv-head, then attention over those blocks.
* ``beam``: per group of beams, the continuations with the highest sums of log
  probabilities over beams and vocabulary.

With ``own`` false everything is computed with elementary torch operations in
fp32 (log probabilities in fp64); with ``own`` true by the library.
"""

import math

import numpy as np
import torch

own = False

BLK = 16                      # tokens a block
E_MIN, E_MAX = -126, 120      # exponents of e4m3 scales
B_MIN, B_MAX = -60, 40        # exponents of bounds and of quantised queries


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # Drafted tokens of a small batch checked in one step: latency counts.
        {"name": "chunk 8 x 5 drafted", "op": "chunk", "kv": "bf16", "nb": 8,
         "Hq": 32, "Hkv": 8, "d": 128, "shared": 0, "ctx_lo": 900,
         "ctx_hi": 3100, "new_lo": 5, "new_hi": 5, "salt": 1},
        # Branches of one tree extended by ragged chunks, the 70B attention shape.
        {"name": "chunk 6 ragged on a tree", "op": "chunk", "kv": "bf16",
         "nb": 6, "Hq": 64, "Hkv": 8, "d": 128, "shared": 4096, "ctx_lo": 1,
         "ctx_hi": 200, "new_lo": 99, "new_hi": 705, "salt": 2},
        # A long prompt.
        {"name": "chunk prompt 1 x 8192", "op": "chunk", "kv": "bf16", "nb": 1,
         "Hq": 64, "Hkv": 8, "d": 128, "shared": 0, "ctx_lo": 0, "ctx_hi": 0,
         "new_lo": 8192, "new_hi": 8192, "salt": 3},
        # Chunks of long requests over an e4m3 pool.
        {"name": "chunk e4m3 4 x ~1000 on ~6000", "op": "chunk", "kv": "e4m3",
         "nb": 4, "Hq": 32, "Hkv": 8, "d": 128, "shared": 0, "ctx_lo": 4001,
         "ctx_hi": 8003, "new_lo": 801, "new_hi": 1203, "salt": 4},
        # One step of mixed requests: single tokens beside chunks, heads of 64.
        {"name": "chunk mixed 24, heads of 64", "op": "chunk", "kv": "bf16",
         "nb": 24, "Hq": 32, "Hkv": 8, "d": 64, "shared": 0, "ctx_lo": 1,
         "ctx_hi": 4000, "new_lo": 1, "new_hi": 512, "mixed": True, "salt": 5},
        # The bounds of a decode step's blocks: latency counts.
        {"name": "bounds step 64 branches", "op": "bounds", "kv": "bf16",
         "nb": 64, "Hkv": 8, "d": 128, "ctx_lo": 1, "ctx_hi": 600, "new_lo": 1,
         "new_hi": 1, "salt": 6},
        # The bounds of prompts that have entered an e4m3 pool, odd lengths.
        {"name": "bounds e4m3 prompts 3 x ~20000", "op": "bounds",
         "kv": "e4m3", "nb": 3, "Hkv": 8, "d": 128, "ctx_lo": 3, "ctx_hi": 90,
         "new_lo": 18001, "new_hi": 22003, "salt": 7},
        # One request with a long context, 2048 of its tokens read.
        {"name": "sparse 1 x 131072", "op": "sparse", "kv": "bf16", "nb": 1,
         "Hq": 64, "Hkv": 8, "d": 128, "lo": 131072, "hi": 131072, "sel": 128,
         "first": 1, "last": 4, "salt": 8},
        # A batch of long contexts.
        {"name": "sparse 32 x ~32000", "op": "sparse", "kv": "bf16", "nb": 32,
         "Hq": 64, "Hkv": 8, "d": 128, "lo": 31001, "hi": 33003, "sel": 128,
         "first": 1, "last": 4, "salt": 9},
        # Requests of mixed lengths over an e4m3 pool, some read whole.
        {"name": "sparse e4m3 48 mixed", "op": "sparse", "kv": "e4m3",
         "nb": 48, "Hq": 32, "Hkv": 8, "d": 128, "lo": 300, "hi": 20000,
         "sel": 96, "first": 4, "last": 2, "salt": 10},
        # One search of eight beams over a small vocabulary: latency counts.
        {"name": "beam 1 x 8, 32000", "op": "beam", "groups": 1, "beams": 8,
         "vocab": 32000, "out": 16, "f32": False, "first": False, "salt": 11},
        # Many searches over a large vocabulary, fp32 logits.
        {"name": "beam 32 x 16, 128256", "op": "beam", "groups": 32,
         "beams": 16, "vocab": 128256, "out": 32, "f32": True, "first": False,
         "salt": 12},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    salt = rng.randrange(1, 1 << 20)
    op = rng.choice(["chunk", "bounds", "sparse", "beam"])
    if op == "beam":
        beams = rng.randrange(1, 17)
        return {"op": op, "groups": log(1, 32), "beams": beams,
                "vocab": log(1000, 128000), "out": rng.randrange(1, 2 * beams + 1),
                "f32": rng.random() < 0.5, "first": rng.random() < 0.2,
                "salt": salt}
    hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "kv": rng.choice(["bf16", "e4m3"]), "Hkv": hkv,
         "d": rng.choice([64, 128]), "salt": salt}
    if op == "bounds":
        step = rng.random() < 0.4
        lo = 1 if step else log(2, 6000)
        return {**c, "nb": log(1, 256) if step else log(1, 8),
                "ctx_lo": rng.randrange(0, 40), "ctx_hi": rng.randrange(40, 700),
                "new_lo": lo, "new_hi": 1 if step else lo + rng.randrange(0, 300)}
    c["Hq"] = hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op == "sparse":
        lo, first, last = log(1, 20000), rng.randrange(0, 5), rng.randrange(1, 5)
        return {**c, "nb": log(1, 32), "lo": lo, "hi": lo + rng.randrange(0, 4000),
                "sel": first + last + log(1, 160), "first": first, "last": last}
    nb = rng.randrange(1, 9)
    lo = log(1, 1200)
    return {**c, "nb": nb, "shared": rng.choice([0, 16 * rng.randrange(1, 128)]),
            "ctx_lo": 0, "ctx_hi": log(1, 4000), "new_lo": lo,
            "new_hi": lo + rng.randrange(0, 300), "mixed": rng.random() < 0.3}


# ---- lengths: a function of the case alone -----------------------------------

def _u(case, what, lo, hi, n):
    g = np.random.default_rng([case["salt"], what])
    return g.integers(lo, hi, size=n, endpoint=True).astype(np.int64)


def _log_u(case, what, lo, hi, n):
    g = np.random.default_rng([case["salt"], what])
    x = np.exp(g.uniform(math.log(lo), math.log(hi), size=n))
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def _lens(case):
    """(cached tokens before the call, new tokens) of every branch; for a sparse
    step (all cached tokens, 1)."""
    nb = case["nb"]
    if case["op"] == "sparse":
        wide = case["hi"] > 10 * case["lo"]
        lens = (_log_u if wide else _u)(case, 0, case["lo"], case["hi"], nb)
        return lens, np.ones(nb, np.int64)
    ctx = _u(case, 0, case["ctx_lo"], case["ctx_hi"], nb) + case.get("shared", 0)
    new = (_log_u if case.get("mixed") else _u)(
        case, 1, case["new_lo"], case["new_hi"], nb)
    return ctx, new


def _layout(case, total_lens):
    """(block tables [nb][max_blocks], blocks of the pool): a shared prefix once,
    everything else apart, in a random physical order."""
    nb = len(total_lens)
    nblk = -(-total_lens // BLK)
    pre = case.get("shared", 0) // BLK if nb > 1 else 0
    blocks = int((nblk - pre).sum()) + pre
    order = np.random.default_rng([case["salt"], 7]).permutation(blocks)
    tables = np.full((nb, int(nblk.max())), -1, np.int32)
    tables[:, :pre] = order[:pre]
    at = pre
    for b in range(nb):
        k = int(nblk[b]) - pre
        tables[b, pre:pre + k] = order[at:at + k]
        at += k
    return tables, blocks


def _vocab_bytes(case):
    return case["groups"] * case["beams"] * case["vocab"] * \
        (4 if case["f32"] else 2)


def work(case):
    op = case["op"]
    if op == "beam":
        rows = case["groups"] * case["beams"]
        return {"bytes": _vocab_bytes(case) + 4 * rows +
                12 * case["groups"] * case["out"],
                "flops": 3 * rows * case["vocab"]}
    ctx, new = _lens(case)
    hkv, d = case["Hkv"], case["d"]
    tile = BLK * d * (1 if case["kv"] == "e4m3" else 2)   # a block's K of a head
    if case["kv"] == "e4m3":
        tile += 8                                         # and its scale
    if op == "bounds":
        nblk = int((-(-(ctx + new) // BLK) - ctx // BLK).sum())
        return {"bytes": nblk * hkv * (tile + 2 * d + 4),
                "flops": 2 * nblk * hkv * BLK * d}
    hq = case["Hq"]
    if op == "sparse":
        nblk = -(-ctx // BLK)
        read = np.minimum(nblk, case["sel"])
        scored = int(np.where(nblk > case["sel"], nblk, 0).sum())
        return {"bytes": hkv * (scored * (2 * d + 4) + int(read.sum()) * 2 * tile) +
                len(ctx) * hq * d * 4 + 4 * hkv * int(read.sum()),
                "flops": hq * d * 4 * (scored + int(read.sum()) * BLK)}
    n = int(new.sum())
    total = ctx + new
    uniq = int(total.sum())
    if case["nb"] > 1:
        uniq -= (case["nb"] - 1) * case["shared"]
    pairs = int((new * ctx + new * (new + 1) // 2).sum())
    return {"bytes": uniq * hkv * 2 * tile // BLK + n * hq * d * 4,
            "flops": 4 * d * hq * pairs}


# ---- inputs ------------------------------------------------------------------

def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["salt"])
    return g


def _pow2(e):
    """2^e in fp32, exactly, e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(amax):
    """Smallest e in range with amax <= 448 * 2^e."""
    m, k = torch.frexp(amax)                 # amax = m 2^k, m in [0.5, 1)
    e = torch.where(m <= 0.875, k - 9, k - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _tile_offsets(d, transposed):
    """Byte of (slot, dimension) in an e4m3 tile, [16][d]."""
    t = torch.arange(BLK, device="cuda")[:, None]
    c = torch.arange(d, device="cuda")[None, :]
    if transposed:
        return c * BLK + t
    return t * d + ((((c >> 4) ^ (t & 7)) << 4) + (c & 15) if d == 128 else c)


def _pieces(n, per):
    """Ranges of n blocks, so that no temporary grows with the pool."""
    step = max(1, (1 << 26) // per)
    return [slice(i, min(i + step, n)) for i in range(0, n, step)]


def _fill_pools(s, g):
    """Keys and values of unit variance, in the pool's type."""
    c = s["case"]
    n, hkv, d = s["blocks"], c["Hkv"], c["d"]
    if c["kv"] == "bf16":
        for k in ("k_pool", "v_pool"):
            s[k] = torch.empty(n, hkv, BLK, d, dtype=torch.bfloat16, device="cuda")
            s[k].normal_(0.0, 1.0, generator=g)
        s["scales"] = None
        return
    s["scales"] = torch.zeros(n, hkv, 4, device="cuda")
    for i, k in enumerate(("k_pool", "v_pool")):
        s[k] = torch.empty(n, hkv, BLK * d, dtype=torch.uint8, device="cuda")
        off = _tile_offsets(d, i == 1).reshape(-1)
        for p in _pieces(n, hkv * BLK * d):
            x = torch.empty(p.stop - p.start, hkv, BLK * d, device="cuda")
            x.normal_(0.0, 1.0, generator=g)
            e = _exponent(x.abs().amax(-1))
            code = (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn)
            s[k][p][:, :, off] = code.view(torch.uint8)
            s["scales"][p, :, i] = _pow2(e)


def prepare(case, seed):
    g = _generator(case, seed)
    s = {"case": case, "seed": seed}
    if case["op"] == "beam":
        n, v = case["groups"] * case["beams"], case["vocab"]
        s["logits"] = torch.empty(
            n, v, dtype=torch.float32 if case["f32"] else torch.bfloat16,
            device="cuda")
        s["logits"].normal_(0.0, 3.0, generator=g)
        # Sums of log probabilities after some twenty tokens; before the first
        # token only one beam of a group counts.
        s["scores"] = torch.empty(n, device="cuda").normal_(-30.0, 2.0, generator=g)
        if case["first"]:
            s["scores"].view(-1, case["beams"])[:, 1:] = -math.inf
        shape = (case["groups"], case["out"])
        s["out_scores"] = torch.zeros(shape, device="cuda")
        s["parents"] = torch.zeros(shape, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.zeros(shape, dtype=torch.int32, device="cuda")
        if own:
            from paged_kv_cache_attn_gb300 import binding as B
            s["ws"] = torch.zeros(
                B.kv_beam_select_workspace_size(case["groups"], case["beams"], v,
                                                case["out"]),
                dtype=torch.uint8, device="cuda")
        return s
    ctx, new = _lens(case)
    total = ctx if case["op"] == "sparse" else ctx + new
    tables, blocks = _layout(case, total)
    nb, n = len(total), int(new.sum())
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s.update({"nb": nb, "n": n, "blocks": blocks, "mb": tables.shape[1],
              "htables": tables, "hlens": total.astype(np.int32),
              "hnew": new.astype(np.int32), "hoff": off,
              "tables": torch.from_numpy(tables).cuda(),
              "lens": torch.from_numpy(total.astype(np.int32)).cuda(),
              "off": torch.from_numpy(off).cuda(),
              "status": torch.zeros(256, dtype=torch.uint8, device="cuda")})
    # A step of one new token a branch needs no offsets.
    s["off_arg"] = None if (new == 1).all() else s["off"]
    _fill_pools(s, g)
    hkv, d = case["Hkv"], case["d"]
    if case["op"] in ("bounds", "sparse"):
        s["bounds"] = torch.zeros(blocks, hkv, 2, d, dtype=torch.int8,
                                  device="cuda")
        s["bscales"] = torch.ones(blocks, hkv, device="cuda")
    if case["op"] == "bounds":
        return s
    hq = case["Hq"]
    s["scale"] = 1.0 / math.sqrt(d)
    s["q"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    s["q"].normal_(0.0, 1.0, generator=g)
    s["out"] = torch.zeros_like(s["q"])
    if case["op"] == "sparse":
        valid = np.zeros(blocks, np.int64)
        for b in range(nb):
            k = -(-int(total[b]) // BLK)
            valid[tables[b, :k]] = np.minimum(BLK, total[b] - BLK * np.arange(k))
        valid = torch.from_numpy(valid).cuda()
        for p in _pieces(blocks, hkv * BLK * d):
            ids = torch.arange(p.start, p.stop, device="cuda")
            s["bounds"][p], s["bscales"][p] = _bounds_of(s, ids, valid[p])
        ns = case["sel"]
        s["sel"] = torch.zeros(nb, hkv, ns, dtype=torch.int32, device="cuda")
        s["sel_tables"] = torch.zeros(nb * hkv, ns, dtype=torch.int32,
                                      device="cuda")
        s["sel_lens"] = torch.zeros(nb * hkv, dtype=torch.int32, device="cuda")
    if own:
        from paged_kv_cache_attn_gb300 import binding as B
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        flags = B.KV_PLAN_KV_E4M3 if case["kv"] == "e4m3" else 0
        if case["op"] == "sparse":
            plan, s["info"] = B.paged_selected_plan(
                nb, hq, hkv, d, s["mb"], s["hlens"], case["sel"], sms, flags)
            s["sel_ws"] = torch.zeros(
                B.paged_select_blocks_workspace_size(nb, s["mb"], hkv),
                dtype=torch.uint8, device="cuda")
        else:
            plan, s["info"] = B.paged_chunk_plan(
                nb, hq, hkv, d, blocks, tables, s["hlens"], s["hnew"], sms, flags)
        s["plan"] = torch.from_numpy(plan).cuda()
        s["ws"] = torch.empty(max(256, s["info"].workspace_bytes),
                              dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _values(s, which, ids):
    """Blocks `ids` of a pool as fp32 [..][Hkv][16][d]."""
    c = s["case"]
    x = s["k_pool" if which == 0 else "v_pool"][ids]
    if c["kv"] == "bf16":
        return x.float()
    off = _tile_offsets(c["d"], which == 1).reshape(-1)
    x = x[..., off].view(torch.float8_e4m3fn).float()
    x = x * s["scales"][ids][..., which, None]
    return x.unflatten(-1, (BLK, c["d"]))


def _bound_exponent(amax):
    """Smallest e in range with amax <= 127 * 2^e."""
    m, k = torch.frexp(amax)
    e = torch.where(m <= 127 / 128, k - 7, k - 6)
    return torch.where(amax > 0, e, torch.full_like(e, B_MIN)).clamp(B_MIN, B_MAX)


def _bounds_of(s, ids, valid):
    """(int8 [n][Hkv][2][d], fp32 [n][Hkv]): bounds of the first `valid` tokens of
    blocks `ids`."""
    k = _values(s, 0, ids)                                    # [n][Hkv][16][d]
    there = (torch.arange(BLK, device="cuda") < valid[:, None])[:, None, :, None]
    lo = torch.where(there, k, math.inf).amin(2)
    hi = torch.where(there, k, -math.inf).amax(2)
    e = _bound_exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    inv = _pow2(-e)[..., None]
    b = torch.stack([torch.floor(lo * inv), torch.ceil(hi * inv)], 2)
    return b.clamp(-127, 127).to(torch.int8), _pow2(e)


def _tokens(s):
    """(branch, position) of every new token."""
    cnt = s["off"][1:] - s["off"][:-1]
    b = torch.repeat_interleave(torch.arange(s["nb"], device="cuda"), cnt.long(),
                                output_size=s["n"])
    i = torch.arange(s["n"], device="cuda") - s["off"][b]
    return b, i, ((s["lens"][b] - cnt[b]) + i).long()


def _plain_bounds(s):
    b, i, pos = _tokens(s)
    # A block once for each of its new tokens: the same result each time.
    lb = pos // BLK
    ids = s["tables"][b, lb].long()
    valid = (s["lens"][b].long() - lb * BLK).clamp(max=BLK)
    first = (i == 0) | (pos % BLK == 0)
    ids, valid = ids[first], valid[first]
    for p in _pieces(len(ids), s["case"]["Hkv"] * BLK * s["case"]["d"]):
        s["bounds"][ids[p]], s["bscales"][ids[p]] = _bounds_of(s, ids[p], valid[p])
    return s["bounds"], s["bscales"]


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_chunk(s):
    c = s["case"]
    hq, hkv, d, nb, n = c["Hq"], c["Hkv"], c["d"], s["nb"], s["n"]
    t = s["tables"].clamp(min=0).long()
    # [nb][Hkv][L][d]; values of slots past a branch's length may be anything.
    k, v = (_values(s, i, t).transpose(1, 2).flatten(2, 3) for i in (0, 1))
    there = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    v = torch.where(there[:, None, :, None], v, 0.0)
    b, i, pos = _tokens(s)
    m = int(s["hnew"].max())
    q = torch.zeros(nb, m, hq, d, device="cuda")
    q[b, i] = s["q"].float() * s["scale"]
    at = torch.zeros(nb, m, dtype=torch.long, device="cuda")
    at[b, i] = pos
    q = q.view(nb, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = q.flatten(2, 3) @ k.transpose(2, 3)                   # [nb][Hkv][G m][L]
    seen = torch.arange(k.shape[2], device="cuda") <= at[:, :, None]
    x.unflatten(2, (-1, m)).masked_fill_(~seen[:, None, None], -math.inf)
    y = (_softmax(x) @ v).unflatten(2, (-1, m))               # [nb][Hkv][G][m][d]
    s["out"].copy_(y.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i])
    return s["out"]


def _quantised(q):
    """Queries as whole numbers of at most 127 times a power of two: the numbers
    in fp32, the power of every head."""
    q = q.float()
    e = _bound_exponent(q.abs().amax(-1))
    return torch.round(q * _pow2(-e)[..., None]).clamp(-127, 127), _pow2(e)


def _plain_select(s):
    c = s["case"]
    nb, hq, hkv, d = s["nb"], c["Hq"], c["Hkv"], c["d"]
    t = s["tables"].clamp(min=0).long()
    bnd = s["bounds"][t].float().permute(0, 2, 1, 3, 4)       # [nb][Hkv][mb][2][d]
    qi, qe = _quantised(s["q"])
    qi = qi.view(nb, hkv, hq // hkv, d)
    # Whole numbers below 2^24: exact in any order.
    x = qi.clamp(max=0) @ bnd[..., 0, :].transpose(2, 3) + \
        qi.clamp(min=0) @ bnd[..., 1, :].transpose(2, 3)
    x = x * qe.view(nb, hkv, -1, 1)
    x = x * s["bscales"][t].transpose(1, 2)[:, :, None]
    x = x.amax(2)                                             # [nb][Hkv][mb]
    j = torch.arange(s["mb"], device="cuda")
    nblk = ((s["lens"] + BLK - 1) // BLK)[:, None]
    always = (j < c["first"]) | (j >= nblk - c["last"])
    x = torch.where(always[:, None], math.inf, x)
    x = torch.where((j < nblk)[:, None], x, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    m = min(c["sel"], s["mb"])
    ids = torch.sort(order[..., :m], -1).values
    # What a branch has too little of comes last.
    ids = torch.where(ids < nblk[..., None], ids, s["mb"])
    ids = torch.sort(ids, -1).values
    s["sel"].fill_(-1)
    s["sel"][..., :m] = torch.where(ids < s["mb"], ids, -1)
    return s["sel"]


def _plain_sparse(s):
    c = s["case"]
    nb, hq, hkv, d = s["nb"], c["Hq"], c["Hkv"], c["d"]
    sel = _plain_select(s).long()
    there = sel >= 0
    ids = torch.gather(s["tables"].long()[:, None].expand(-1, hkv, -1), 2,
                       sel.clamp(min=0)).clamp(min=0)         # physical
    h = torch.arange(hkv, device="cuda")[None, :, None].expand_as(ids)
    if c["kv"] == "bf16":
        k, v = s["k_pool"][ids, h].float(), s["v_pool"][ids, h].float()
    else:
        k, v = (_e4m3_tiles(s, i, ids, h) for i in (0, 1))
    k, v = k.flatten(2, 3), v.flatten(2, 3)                   # [nb][Hkv][T][d]
    tok = sel[..., None] * BLK + torch.arange(BLK, device="cuda")
    seen = (there[..., None] & (tok < s["lens"][:, None, None, None])).flatten(2)
    q = (s["q"].float() * s["scale"]).view(nb, hkv, hq // hkv, d)
    x = torch.where(seen[:, :, None], q @ k.transpose(2, 3), -math.inf)
    y = _softmax(x) @ torch.where(seen[..., None], v, 0.0)
    s["out"].copy_(y.view(nb, hq, d))
    return s["out"], s["sel"]


def _e4m3_tiles(s, which, ids, h):
    off = _tile_offsets(s["case"]["d"], which == 1).reshape(-1)
    x = s["k_pool" if which == 0 else "v_pool"][ids, h][..., off]
    x = x.view(torch.float8_e4m3fn).float() * s["scales"][ids, h, which][..., None]
    return x.unflatten(-1, (BLK, -1))


def _plain_beam(s):
    c = s["case"]
    n, beams = c["out"], c["beams"]
    x = s["logits"].float()
    # Per beam: keys that order by logit, then by lower token.
    u = x.view(torch.int32).long()
    u = torch.where(u >= 0, u, -(u & 0x7fffffff))
    tok = torch.arange(c["vocab"], device="cuda")
    key = torch.topk(u * (1 << 32) - tok, min(n, c["vocab"]), dim=1).values
    tok = (-key) % (1 << 32)
    x = x.double()
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    y = s["scores"].double()[:, None] + (torch.gather(x, 1, tok) - lse)
    y = y.view(c["groups"], -1)
    best, at = torch.sort(y, dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    s["out_scores"].copy_(best)
    s["parents"].copy_(at // key.shape[1])
    s["tokens"].copy_(torch.gather(tok.view(c["groups"], -1), 1, at))
    return s["out_scores"], s["parents"], s["tokens"]


_run_plain = {"chunk": _plain_chunk, "bounds": _plain_bounds,
              "sparse": _plain_sparse, "beam": _plain_beam}


# ---- the library's calls -----------------------------------------------------

def _own_chunk(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    tail = (s["blocks"], s["n"], s["nb"], c["Hq"], c["Hkv"], c["d"], s["scale"],
            s["out"], s["plan"], s["info"], s["ws"], s["ws"].numel())
    if c["kv"] == "bf16":
        B.paged_chunk_attn(s["q"], s["k_pool"], s["v_pool"], *tail)
    else:
        B.paged_chunk_attn_e4m3(s["q"], s["k_pool"], s["v_pool"], s["scales"],
                                *tail)
    return s["out"]


def _own_bounds(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    tail = (s["blocks"], s["tables"], s["lens"], s["off_arg"], s["n"], s["nb"],
            s["mb"], c["Hkv"], c["d"], s["bounds"], s["bscales"], s["status"])
    if c["kv"] == "bf16":
        B.paged_key_bounds(s["k_pool"], *tail)
    else:
        B.paged_key_bounds_e4m3(s["k_pool"], s["scales"], *tail)
    return s["bounds"], s["bscales"]


def _own_sparse(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    B.paged_select_blocks(
        s["q"], s["bounds"], s["bscales"], s["blocks"], s["tables"], s["lens"],
        s["nb"], s["mb"], c["Hq"], c["Hkv"], c["d"], c["sel"], c["first"],
        c["last"], s["sel"], s["sel_tables"], s["sel_lens"], s["sel_ws"])
    tail = (s["blocks"], s["sel_tables"], s["sel_lens"], s["nb"], c["Hq"],
            c["Hkv"], c["d"], c["sel"], s["scale"], s["out"], s["plan"],
            s["info"], s["ws"], s["ws"].numel())
    if c["kv"] == "bf16":
        B.paged_selected_attn(s["q"], s["k_pool"], s["v_pool"], *tail)
    else:
        B.paged_selected_attn_e4m3(s["q"], s["k_pool"], s["v_pool"], s["scales"],
                                   *tail)
    return s["out"], s["sel"]


def _own_beam(s):
    from paged_kv_cache_attn_gb300 import binding as B
    c = s["case"]
    B.kv_beam_select(s["logits"], s["scores"], c["groups"], c["beams"], c["out"],
                     s["out_scores"], s["parents"], s["tokens"], s["ws"])
    return s["out_scores"], s["parents"], s["tokens"]


_run_own = {"chunk": _own_chunk, "bounds": _own_bounds, "sparse": _own_sparse,
            "beam": _own_beam}


# ---- the definition in 64 bits -----------------------------------------------

def _exact_rows(s, which, b, h=None):
    """Cached keys or values of a branch in float64: [L][Hkv][d]."""
    c = s["case"]
    L = int(s["hlens"][b])
    ids = torch.from_numpy(s["htables"][b, :-(-L // BLK)].astype(np.int64)).cuda()
    x = s["k_pool" if which == 0 else "v_pool"][ids]
    if c["kv"] == "e4m3":
        val = x.view(torch.float8_e4m3fn).double()
        if which == 1:
            val = val.unflatten(-1, (c["d"], BLK)).transpose(2, 3)
        else:
            val = val.unflatten(-1, (BLK, c["d"]))
            if c["d"] == 128:
                # Chunk i of row t lies at chunk i ^ (t mod 8).
                t = torch.arange(BLK, device="cuda")[:, None] % 8
                at = torch.arange(8, device="cuda")[None] ^ t
                val = torch.gather(
                    val.unflatten(-1, (8, 16)), 3,
                    at[None, None, :, :, None].expand(*val.shape[:2], -1, -1, 16)
                ).flatten(3)
        x = val * s["scales"][ids][..., which].double()[..., None, None]
    return x.double().transpose(1, 2).flatten(0, 1)[:L]


def _exact_pow2(e):
    """2^e in float64 from its bits (a power function need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_exponent(amax):
    """Smallest e in [B_MIN, B_MAX] with amax <= 127 * 2^e, by trying each."""
    lim = 127.0 * _exact_pow2(torch.arange(B_MIN, B_MAX + 1, device="cuda"))
    return B_MIN + (amax[..., None] > lim[:-1]).sum(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "beam":
        g, n, v = case["groups"], case["out"], case["vocab"]
        y = torch.empty(g, case["beams"] * v, dtype=torch.float64, device="cuda")
        for i in range(g):
            x = s["logits"].view(g, -1, v)[i].double()
            y[i] = (s["scores"].view(g, -1)[i].double()[:, None] +
                    torch.log_softmax(x, 1)).flatten()
        out = [torch.empty(g, n, dtype=torch.float64, device="cuda")]
        out += [torch.empty(g, n, dtype=torch.int32, device="cuda") for _ in "pt"]
        for i in range(g):
            best, at = torch.sort(y[i], dim=0, descending=True, stable=True)
            out[0][i], out[1][i], out[2][i] = best[:n], at[:n] // v, at[:n] % v
        return tuple(out)
    hkv, d = case["Hkv"], case["d"]
    if op == "bounds":
        bnd, sc = s["bounds"].clone(), s["bscales"].double()
        for b in range(s["nb"]):
            k = _exact_rows(s, 0, b)
            L, new = int(s["hlens"][b]), int(s["hnew"][b])
            lb = (L - new) // BLK
            k = k[lb * BLK:]
            ids = torch.from_numpy(
                s["htables"][b, lb:-(-L // BLK)].astype(np.int64)).cuda()
            pad = len(ids) * BLK - len(k)
            # Repeats of a block's last token leave its bounds.
            k = torch.cat([k, k[-1:].expand(pad, -1, -1)]).view(-1, BLK, hkv, d)
            lo, hi = k.amin(1), k.amax(1)
            p = _exact_pow2(_exact_exponent(torch.maximum(-lo, hi).amax(-1)))
            lo = torch.floor(lo / p[..., None]).clamp(-127, 127)
            hi = torch.ceil(hi / p[..., None]).clamp(-127, 127)
            bnd[ids, :, 0], bnd[ids, :, 1] = lo.to(torch.int8), hi.to(torch.int8)
            sc[ids] = p
        return bnd, sc
    hq = case["Hq"]
    grp = hq // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    sel = None
    if op == "sparse":
        sel = torch.full(s["sel"].shape, -1, dtype=torch.int32, device="cuda")
    for b in range(s["nb"]):
        L, m = int(s["hlens"][b]), int(s["hnew"][b])
        k, v = _exact_rows(s, 0, b), _exact_rows(s, 1, b)
        if op == "chunk":
            see = torch.ones(m, L, dtype=torch.bool, device="cuda").tril(L - m)
            rows = slice(int(s["hoff"][b]), int(s["hoff"][b + 1]))
            for h in range(hq):
                x = s["q"][rows, h].double() @ k[:, h // grp].T * s["scale"]
                x[~see] = -math.inf
                out[rows, h] = torch.softmax(x, -1) @ v[:, h // grp]
            continue
        nblk = -(-L // BLK)
        ids = torch.from_numpy(s["htables"][b, :nblk].astype(np.int64)).cuda()
        for g in range(hkv):
            q = s["q"][b, g * grp:(g + 1) * grp].double()
            pick = torch.arange(nblk, device="cuda")
            if nblk > case["sel"]:
                p = _exact_pow2(_exact_exponent(q.abs().amax(-1)))
                qi = torch.round(q / p[:, None]).clamp(-127, 127)
                bd = s["bounds"][ids, g].double()             # [nblk][2][d]
                x = torch.maximum(qi[:, None] * bd[:, 0], qi[:, None] * bd[:, 1])
                x = x.sum(-1) * p[:, None] * s["bscales"][ids, g].double()
                x = x.amax(0)
                x[:case["first"]] = math.inf
                x[nblk - case["last"]:] = math.inf
                pick = torch.sort(x, dim=0, descending=True, stable=True).indices
                pick = pick[:case["sel"]].sort().values
            sel[b, g, :len(pick)] = pick.int()
            tok = (pick[:, None] * BLK + torch.arange(BLK, device="cuda")).flatten()
            tok = tok[tok < L]
            x = q @ k[tok, g].T * s["scale"]
            out[b, g * grp:(g + 1) * grp] = torch.softmax(x, -1) @ v[tok, g]
    return out if op == "chunk" else (out, sel)
