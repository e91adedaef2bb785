"""Rotating appends of decode steps, one new token a branch without row_offsets:
the values of paged_rope_append_e4m3 against the rotation in 64 bits, and the same
call as a chunk of one token a branch."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import _rope_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402
from test_gpu_rope import HALVES, PAIRS, gen, make_cache, snapshot  # noqa: E402

CONTEXTS = {
    "one": [0],
    "edges": [0, 1, 14, 15, 16, 17, 31, 32, 100],
    "many": [(37 * i) % 61 for i in range(90)],
}


def codes(c, which, d):
    """[blocks][Hkv][16][d] values of K or V, in 64 bits, without their scales."""
    x = (c.k if which == 0 else c.v)[0].view(torch.float8_e4m3fn).double()
    x = x.flatten(-1).view(x.shape[0], x.shape[1], 16 * d)
    t = torch.arange(16, device="cuda")[:, None]
    ch = torch.arange(d, device="cuda")[None, :]
    if which == 1:
        at = ch * 16 + t
    elif d == 128:
        at = t * 128 + (((ch >> 4) ^ (t & 7)) << 4) + (ch & 15)
    else:
        at = t * d + ch
    return x[..., at]


@pytest.mark.parametrize("name", list(CONTEXTS))
@pytest.mark.parametrize("style,Hq,Hkv,d,rot", [
    (HALVES, 4, 1, 128, 128), (PAIRS, 32, 8, 128, 64), (HALVES, 3, 3, 64, 32),
    (PAIRS, 130, 2, 64, 64), (HALVES, 40, 40, 128, 48)])
def test_rope_step_e4m3(name, style, Hq, Hkv, d, rot):
    """Half an e4m3 step (2^-4 of the value, or half of the smallest step, 2^-10 of
    the scale) and the fp32 arithmetic before it; the scale is the smallest that
    fits the block's first token, or the block's own unless the token needs more;
    stored rows are rounded once more where it grew."""
    ctx = CONTEXTS[name]
    ids, nb = list(range(len(ctx))), len(ctx)
    a, b = (make_cache("e4m3", ctx, Hq, Hkv, d) for _ in range(2))
    rn = gen(17)
    # Some tokens need a larger scale than the rows that are there.
    gain = torch.tensor([0.2, 3.0, 40.0], device="cuda")[
        torch.arange(nb, device="cuda") % 3][:, None, None]
    qkv = rn(nb, (Hq + 2 * Hkv) * d)
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = (qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)) * gain).bfloat16()
    v = (qkv[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)) * gain).bfloat16()
    tab = R.table(max(ctx) + 1, rot).cuda()
    bt = {}
    for c in (a, b):
        B.kv_reserve(c.h, ids, [1] * nb)
        bt[c] = c.batch(ids).upload()
    old = [x.clone() for x in (codes(a, 0, d), codes(a, 1, d), a.scales[0])]
    before = snapshot(a)
    qo = torch.full((nb + 1, Hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    bt[a].append_rotated(q, k, v, tab, style, qo[:nb])
    assert bt[a].append_status() == (0, 0)
    pos = torch.tensor(ctx, device="cuda")
    y, mag = R.rotate(q, tab, pos, style == PAIRS)
    assert ((qo[:nb].double() - y).abs() <= R.bf16_bound(y, mag)).all()
    assert (qo[nb] == 7).all()
    phys = torch.from_numpy(
        bt[a].tables[np.arange(nb), np.array(ctx) // 16].astype(np.int64)).cuda()
    slot = pos % 16
    new_scale = a.scales[0].double()
    for which, x in ((0, k), (1, v)):
        if which == 0:
            want, mag = R.rotate(x, tab, pos, style == PAIRS)
        else:
            want, mag = x.double(), torch.zeros_like(x, dtype=torch.float64)
        got = codes(a, which, d)
        sc = new_scale[phys, :, which]                       # [nb][Hkv]
        val = got[phys, :, slot] * sc[..., None]
        lim = want.abs() * 2.0 ** -4 + sc[..., None] * 2.0 ** -10 + mag * 2.0 ** -22
        assert ((val - want).abs() <= lim).all()
        # The scale.
        amax = want.abs().amax(-1)
        was = old[2][phys, :, which].double()
        first = (slot == 0)[:, None]
        assert (amax <= 448 * sc * (1 + 2.0 ** -20)).all()
        tight = amax > 224 * sc * (1 - 2.0 ** -20)
        assert (tight | (~first & (sc == was))).all()
        assert (first | (sc >= was)).all()
        # Rows stored before.
        rows = torch.arange(16, device="cuda")[None, None, :, None] < \
            slot[:, None, None, None]
        then = old[which][phys] * was[..., None, None]
        now = got[phys] * sc[..., None, None]
        grew = (sc != was)[..., None, None]
        lim = torch.where(grew, then.abs() * 2.0 ** -4 +
                          sc[..., None, None] * 2.0 ** -10, 0.0)
        assert (~rows | ((now - then).abs() <= lim)).all()
    # Other blocks as they were.
    rest = torch.ones(a.k.shape[1], dtype=torch.bool, device="cuda")
    rest[phys] = False
    for x, z in zip((a.k, a.v, a.scales), before):
        assert torch.equal(x[0][rest], z[0][rest])
    # The same tokens as chunks of one.
    off = torch.arange(nb + 1, dtype=torch.int32, device="cuda")
    q2 = torch.empty_like(qo[:nb])
    bt[b].append_rotated(q, k, v, tab, style, q2, off)
    assert bt[b].append_status() == (0, 0)
    assert torch.equal(q2, qo[:nb])
    assert torch.equal(a.scales[0][phys][..., :2], b.scales[0][phys][..., :2])
    upto = torch.arange(16, device="cuda")[None, None, :, None] <= \
        slot[:, None, None, None]
    for which in (0, 1):
        x, z = codes(a, which, d)[phys], codes(b, which, d)[phys]
        assert (~upto | (x == z)).all()
    a.close()
    b.close()


def test_rope_step_e4m3_keys_alone_and_in_place():
    """Without queries, and with queries rotated where they are."""
    ctx = CONTEXTS["edges"]
    ids, nb = list(range(len(ctx))), len(ctx)
    caches = [make_cache("e4m3", ctx, 8, 2, 128) for _ in range(3)]
    rn = gen(19)
    q, k, v = rn(nb, 8, 128), rn(nb, 2, 128), rn(nb, 2, 128)
    tab = R.table(200, 128).cuda()
    out, outs = torch.empty_like(q), []
    for c, (src, dst) in zip(caches, ((None, None), (q, out), (q, q))):
        B.kv_reserve(c.h, ids, [1] * nb)
        bt = c.batch(ids).upload()
        bt.append_rotated(src, k, v, tab, HALVES, dst)
        assert bt.append_status() == (0, 0)
        phys = torch.from_numpy(
            bt.tables[np.arange(nb), np.array(ctx) // 16].astype(np.int64)).cuda()
        slot = torch.tensor(ctx, device="cuda") % 16
        outs.append([codes(c, w, 128)[phys, :, slot] for w in (0, 1)] +
                    [c.scales[0][phys][..., :2].clone()])
    assert torch.equal(out, q)
    for o in outs[1:]:
        for x, z in zip(outs[0], o):
            assert torch.equal(x, z)
    for c in caches:
        c.close()
