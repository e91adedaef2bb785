"""paged_rope_append, paged_rope_append_e4m3 and paged_latent_append on the GPU.

Rotated values against the rotation in 64 bits within one rounding to bf16
(plus the fp32 arithmetic before it); with a table of zero angles the pools
equal, bit for bit, what kv_append_batch leaves; values outside the written
slots are left as they were.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import _rope_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402
from paged_kv_cache_attn_gb300 import harness as H  # noqa: E402
from paged_kv_cache_attn_gb300 import workloads as W  # noqa: E402

HALVES, PAIRS = B.KV_ROPE_HALVES, B.KV_ROPE_PAIRS


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda",
                                  dtype=torch.float32).bfloat16()


def make_cache(kv, ctx, Hq, Hkv, d, fan=0):
    """Independent branches of the given lengths; fan > 0: one root of ctx[0]
    tokens forked fan times, nothing appended (partial blocks copied)."""
    w = W.Workload("rope", Hq, Hkv, d, 77)
    if fan:
        w.nodes = [W.NodeSpec(-1, ctx[0])] + [W.NodeSpec(0, 0)] * fan
        w.ops = [("create",), ("append", 0), ("fork", 0, fan)]
    else:
        for i, n in enumerate(ctx):
            w.nodes.append(W.NodeSpec(-1, int(n)))
            w.ops += [("create",), ("append", i)]
    w.num_blocks = 400
    c = H.Cache(w, kv_dtype=kv)
    torch.cuda.synchronize()
    return c


def snapshot(c):
    t = [c.k.clone(), c.v.clone()]
    return t + ([c.scales.clone()] if c.scales is not None else [])


CHUNKS = [
    # (contexts, new tokens)
    ([0], [1]),
    ([15, 16, 17, 0], [1, 1, 1, 1]),
    ([0, 5, 31, 16], [16, 11, 18, 40]),
    ([7, 100, 0], [0, 37, 129]),
    ([3] * 40, [2] * 40),
]


@pytest.mark.parametrize("ctx,new", CHUNKS)
@pytest.mark.parametrize("style", [HALVES, PAIRS])
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(4, 2, 64, 64), (5, 1, 128, 128),
                                          (32, 8, 128, 64), (3, 3, 64, 16),
                                          (8, 4, 128, 48)])
def test_rope_append_bf16(ctx, new, style, Hq, Hkv, d, rot):
    c = make_cache("bf16", ctx, Hq, Hkv, d)
    ids = list(range(len(ctx)))
    B.kv_reserve(c.h, ids, new)
    live = [i for i in ids if ctx[i] + new[i] > 0]
    assert live == ids
    bt = c.batch(ids).upload()
    n = sum(new)
    rn = gen(5)
    qkv = rn(n, (Hq + 2 * Hkv) * d + 8)            # a row wider than its parts
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = qkv[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].unflatten(1, (Hkv, d))
    qo = torch.full((n + 1, Hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    tab = R.table(max(a + b for a, b in zip(ctx, new)), rot).cuda()
    off = None if all(x == 1 for x in new) else torch.tensor(
        np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    before = snapshot(c)
    bt.append_rotated(q, k, v, tab, style, qo[:n], off)
    torch.cuda.synchronize()
    assert bt.append_status() == (0, 0)
    br, pos = R.positions([int(x) for x in bt.seq_lens], new)
    p = torch.from_numpy(pos).cuda()
    y, mag = R.rotate(q, tab, p, style == PAIRS)
    assert ((qo[:n].double() - y).abs() <= R.bf16_bound(y, mag)).all()
    assert torch.equal(qo[n], torch.full_like(qo[n], 7.0))
    y, mag = R.rotate(k, tab, p, style == PAIRS)
    phys = torch.from_numpy(bt.tables[br, pos // 16].astype(np.int64)).cuda()
    slot = p % 16
    assert ((c.k[0][phys, :, slot].double() - y).abs()
            <= R.bf16_bound(y, mag)).all()
    assert torch.equal(c.v[0][phys, :, slot], v)
    # Everything else as it was.
    before[0][0][phys, :, slot] = c.k[0][phys, :, slot]
    before[1][0][phys, :, slot] = c.v[0][phys, :, slot]
    assert torch.equal(before[0].view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(before[1].view(torch.int16), c.v.view(torch.int16))
    c.close()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,new", CHUNKS)
@pytest.mark.parametrize("Hkv,d,style", [(2, 64, HALVES), (1, 128, PAIRS),
                                         (8, 128, HALVES)])
def test_zero_angles_equal_a_plain_append(kv, ctx, new, Hkv, d, style):
    a = make_cache(kv, ctx, Hkv, Hkv, d)
    b = make_cache(kv, ctx, Hkv, Hkv, d)
    ids = list(range(len(ctx)))
    n = sum(new)
    rn = gen(9)
    # Growing values, so that a later write needs a larger scale than the rows
    # already stored; and a row of zeros.
    k = rn(n, Hkv, d) * torch.linspace(0.5, 90, n, device="cuda")[:, None, None]
    v = rn(n, Hkv, d) * torch.linspace(64, 0, n, device="cuda")[:, None, None]
    k, v = k.bfloat16(), v.bfloat16()
    B.kv_append_batch(a.h, ids, new, k, v)
    B.kv_reserve(b.h, ids, new)
    bt = b.batch(ids).upload()
    tab = torch.zeros(max(int(x) for x in bt.seq_lens), d // 2, 2, device="cuda")
    tab[..., 0] = 1.0
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]),
                       dtype=torch.int32, device="cuda")
    bt.append_rotated(None, k, v, tab, style, None, off)
    torch.cuda.synchronize()
    assert bt.append_status() == (0, 0)
    assert a.tables() == b.tables()
    for i in ids:
        t, L = B.kv_get_block_table(a.h, i)
        t = torch.from_numpy(t.astype(np.int64)).cuda()
        if kv == "bf16":
            x = [p[0][t].transpose(1, 2).flatten(0, 1)[:L] for p in (a.k, a.v, b.k, b.v)]
            assert torch.equal(x[0].view(torch.int16), x[2].view(torch.int16))
            assert torch.equal(x[1].view(torch.int16), x[3].view(torch.int16))
        else:
            assert torch.equal(a.scales[0][t][..., :2], b.scales[0][t][..., :2])
            kk = a.k[0][t] == b.k[0][t]
            vv = a.v[0][t] == b.v[0][t]
            # Bytes of slots past the length hold whatever they held.
            m = L - 16 * (len(t) - 1)
            if m < 16 and len(t):
                kk[-1] |= (torch.arange(16 * d, device="cuda") // d >= m)
                vv[-1] |= (torch.arange(16 * d, device="cuda") % 16 >= m)
            assert kk.all() and vv.all()
    a.close()
    b.close()


@pytest.mark.parametrize("ctx,new", CHUNKS)
@pytest.mark.parametrize("style,d,rot", [(HALVES, 128, 128), (PAIRS, 128, 64),
                                         (HALVES, 64, 32), (PAIRS, 64, 64)])
def test_rope_append_e4m3(ctx, new, style, d, rot):
    """The stored value code * scale is within half an e4m3 step of the
    rotated key (2^-4 relative, or half of the smallest step 2^-9), the scale
    the smallest that fits, rows already stored within one more rounding."""
    Hq, Hkv = 4, 2
    c = make_cache("e4m3", ctx, Hq, Hkv, d)
    ids = list(range(len(ctx)))
    B.kv_reserve(c.h, ids, new)
    bt = c.batch(ids).upload()
    n = sum(new)
    rn = gen(11)
    q, k, v = rn(n, Hq, d), rn(n, Hkv, d) * 3, rn(n, Hkv, d)
    qo = torch.empty_like(q)
    tab = R.table(max(int(x) for x in bt.seq_lens), rot).cuda()
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]),
                       dtype=torch.int32, device="cuda")
    old_scale = c.scales.clone()
    old_k = c.k.clone()
    bt.append_rotated(q, k, v, tab, style, qo, off)
    torch.cuda.synchronize()
    assert bt.append_status() == (0, 0)
    br, pos = R.positions([int(x) for x in bt.seq_lens], new)
    p = torch.from_numpy(pos).cuda()
    y, mag = R.rotate(q, tab, p, style == PAIRS)
    assert ((qo.double() - y).abs() <= R.bf16_bound(y, mag)).all()
    y, mag = R.rotate(k, tab, p, style == PAIRS)
    y, mag = y.cpu(), mag.cpu()

    def tile(codes, scale, phys, h):
        x = codes[0, phys, h].view(torch.float8_e4m3fn).double().cpu() \
            .view(16, d)
        if d == 128:
            t = torch.arange(16)[:, None]
            ch = torch.arange(d)[None, :]
            x = x.view(-1)[t * 128 + (((ch >> 4) ^ (t & 7)) << 4) + (ch & 15)]
        return x * scale[0, phys, h, 0].double().cpu()

    for i in ids:
        t, L = B.kv_get_block_table(c.h, i)
        for lb in range(ctx[i] // 16, len(t)):
            phys = int(t[lb])
            rows = np.nonzero((br == i) & (pos // 16 == lb))[0]
            if not len(rows):
                continue
            s0 = int(pos[rows[0]]) % 16
            for h in range(Hkv):
                sc = float(c.scales[0, phys, h, 0])
                want = y[rows, h]
                got = tile(c.k, c.scales, phys, h)
                e = want.abs() * 2.0 ** -4 + sc * 2.0 ** -10 + mag[rows, h] * 2.0 ** -22
                assert ((got[s0:s0 + len(rows)] - want).abs() <= e).all()
                amax = float(want.abs().max())
                assert amax <= 448 * sc * (1 + 2.0 ** -20)
                if s0 == 0:
                    assert amax > 224 * sc * (1 - 2.0 ** -20)
                else:
                    o = float(old_scale[0, phys, h, 0])
                    assert sc >= o and (sc == o or amax > 224 * sc * (1 - 2.0 ** -20))
                    was = tile(old_k, old_scale, phys, h)[:s0]
                    d2 = (got[:s0] - was).abs()
                    lim = 0 if sc == o else was.abs() * 2.0 ** -4 + sc * 2.0 ** -10
                    assert (d2 <= lim).all()
    c.close()


@pytest.mark.parametrize("ctx,new", CHUNKS)
@pytest.mark.parametrize("style", [HALVES, PAIRS])
@pytest.mark.parametrize("Hq", [1, 16, 130])
def test_latent_append(ctx, new, style, Hq):
    c = make_cache("latent", ctx, Hq, 1, 512)
    ids = list(range(len(ctx)))
    B.kv_reserve(c.h, ids, new)
    bt = c.batch(ids).upload()
    n = sum(new)
    rn = gen(3)
    row = rn(n, 576)
    q = rn(n, Hq, 192)
    before_q = q.clone()
    qa = torch.full((n, Hq, 576), 5.0, device="cuda", dtype=torch.bfloat16)
    tab = R.table(max(int(x) for x in bt.seq_lens), 64).cuda()
    off = None if all(x == 1 for x in new) else torch.tensor(
        np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    snap = snapshot(c)
    bt.append_rotated(q[..., 128:], row[:, :512], row[:, 512:], tab, style,
                      qa[..., 512:], off)
    torch.cuda.synchronize()
    assert bt.append_status() == (0, 0)
    br, pos = R.positions([int(x) for x in bt.seq_lens], new)
    p = torch.from_numpy(pos).cuda()
    y, mag = R.rotate(q[..., 128:], tab, p, style == PAIRS)
    assert ((qa[..., 512:].double() - y).abs() <= R.bf16_bound(y, mag)).all()
    assert (qa[..., :512] == 5).all()
    phys = torch.from_numpy(bt.tables[br, pos // 16].astype(np.int64)).cuda()
    slot = p % 16
    y, mag = R.rotate(row[:, None, 512:], tab, p, style == PAIRS)
    got = c.v[0][phys, 0, slot].double()
    assert ((got - y[:, 0]).abs() <= R.bf16_bound(y, mag)[:, 0]).all()
    assert torch.equal(c.k[0][phys, 0, slot], row[:, :512])
    snap[0][0][phys, 0, slot] = c.k[0][phys, 0, slot]
    snap[1][0][phys, 0, slot] = c.v[0][phys, 0, slot]
    assert torch.equal(snap[0].view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(snap[1].view(torch.int16), c.v.view(torch.int16))
    # In place, the same result; and again from the same inputs.
    bt.append_rotated(q[..., 128:], row[:, :512], row[:, 512:], tab, style,
                      q[..., 128:], off)
    assert torch.equal(q[..., 128:], qa[..., 512:])
    assert torch.equal(q[..., :128], before_q[..., :128])
    c.close()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "latent"])
def test_bad_tokens_are_recorded_and_skipped(kv):
    """A position past the table, and a table entry past the pool: recorded,
    nothing written for those tokens, the others written."""
    d, Hkv = (512, 1) if kv == "latent" else (64, 1)
    c = make_cache(kv, [20, 5, 40], 2, Hkv, d)
    B.kv_reserve(c.h, [0, 1, 2], [1, 1, 1])
    bt = c.batch([0, 1, 2]).upload()
    rn = gen(1)
    k = rn(3, 512) if kv == "latent" else rn(3, Hkv, d)
    v = rn(3, 64) if kv == "latent" else rn(3, Hkv, d)
    q = rn(3, 2, 64)
    qo = torch.full_like(q, 9.0)
    tab = R.table(30, 64).cuda()               # branch 2 sits at position 40
    snap = snapshot(c)
    bt.append_rotated(q, k, v, tab, HALVES, qo)
    assert bt.append_status() == (B.KV_ERR_DEVICE, 40)
    assert bt.append_status() == (0, 0)
    assert (qo[2] == 9).all() and not (qo[:2] == 9).all(-1).any()
    t2 = int(bt.tables[2, 2])
    assert torch.equal(c.k[0, t2].view(torch.uint8), snap[0][0, t2].view(torch.uint8))
    bt.dev["tables"][0, 1] = c.w.num_blocks + 3
    bt.dev["tables"][2, 2] = -7
    snap = snapshot(c)
    tab = R.table(64, 64).cuda()
    bt.append_rotated(q, k, v, tab, HALVES, qo)
    code, detail = bt.append_status()
    assert code == B.KV_ERR_DEVICE and detail in (c.w.num_blocks + 3, -7)
    for blk in range(c.w.num_blocks):
        if blk != int(bt.tables[1, 0]):
            assert torch.equal(c.k[0, blk].view(torch.uint8),
                               snap[0][0, blk].view(torch.uint8))
    c.close()


def test_steps_in_a_graph_on_a_side_stream():
    """Two graphs captured on side streams, each with its own buffers, replayed
    in turn with new inputs."""
    c = make_cache("bf16", [10, 33, 16], 4, 2, 128)
    B.kv_reserve(c.h, [0, 1, 2], [1, 1, 1])
    bt = c.batch([0, 1, 2]).upload()
    tab = R.table(64, 128).cuda()
    rn = gen(2)
    q, k, v = rn(3, 4, 128), rn(3, 2, 128), rn(3, 2, 128)
    qo = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bt.append_rotated(q, k, v, tab, PAIRS, qo)
    for seed in (4, 5):
        x = gen(seed)
        q.copy_(x(3, 4, 128))
        k.copy_(x(3, 2, 128))
        v.copy_(x(3, 2, 128))
        g.replay()
        torch.cuda.synchronize()
        p = torch.tensor([10, 33, 16], device="cuda")
        y, mag = R.rotate(q, tab, p, True)
        assert ((qo.double() - y).abs() <= R.bf16_bound(y, mag)).all()
    c.close()
