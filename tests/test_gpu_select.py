"""Bounds of blocks' keys, selection by them and the decode step over what was
selected, against their definitions in 64 bits."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _chunk_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


def pow2(e):
    """2^e in float64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exponent(amax):
    e = torch.arange(-60, 41, device=amax.device)
    return -60 + (amax[..., None] > 127.0 * pow2(e)[:-1]).sum(-1)


def bounds_of(k):
    """k [tokens][Hkv][d] of one block: (int8 [Hkv][2][d], scale [Hkv])."""
    odd = ~k.isfinite().all(0).all(-1)
    k = torch.where(odd[:, None], 0.0, k)
    lo, hi = k.amin(0), k.amax(0)
    p = pow2(exponent(torch.maximum(-lo, hi).amax(-1)))
    b = torch.stack([torch.floor(lo / p[:, None]), torch.ceil(hi / p[:, None])], 1)
    b = torch.where(odd[:, None, None], 0.0, b.clamp(-127, 127))
    return b.to(torch.int8), torch.where(odd, math.inf, p)


class Tree:
    """Branches of `lens` tokens in a pool of random blocks."""

    def __init__(self, Hq, Hkv, d, lens, kv="bf16", seed=1, spare=2):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.kv = Hq, Hkv, d, kv
        self.lens = np.array(lens, np.int32)
        self.nb = len(lens)
        nblk = -(-self.lens // 16)
        self.mb = max(1, int(nblk.max()))
        self.blocks = int(nblk.sum()) + spare
        order = rng.permutation(self.blocks)
        self.tables = np.full((self.nb, self.mb), -1, np.int32)
        at = 0
        for b in range(self.nb):
            self.tables[b, :nblk[b]] = order[at:at + nblk[b]]
            at += nblk[b]
        self.k, self.v, self.scales, self.kx, self.vx = R.pool(
            self.blocks, Hkv, d, self.g, kv)
        self.dt = torch.from_numpy(self.tables).cuda()
        self.dl = torch.from_numpy(self.lens).cuda()
        self.bounds = torch.full((self.blocks, Hkv, 2, d), 99, dtype=torch.int8,
                                 device="cuda")
        self.bscales = torch.full((self.blocks, Hkv), 99.0, device="cuda")
        self.status = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.q = torch.randn(self.nb, Hq, d, generator=self.g,
                             device="cuda").bfloat16()

    def update(self, new=None):
        """Bounds of the blocks with the last new[b] tokens (None: one each)."""
        off, total = None, self.nb
        if new is not None:
            off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            total = int(off[-1])
            off = torch.from_numpy(off).cuda()
        tail = (self.blocks, self.dt, self.dl, off, total, self.nb, self.mb,
                self.Hkv, self.d, self.bounds, self.bscales, self.status)
        if self.kv == "bf16":
            B.paged_key_bounds(self.k, *tail)
        else:
            B.paged_key_bounds_e4m3(self.k, self.scales, *tail)
        assert B.kv_check_device_status(self.status) == (0, 0)

    def check_bounds(self, new=None):
        want_b = torch.full_like(self.bounds, 99)
        want_s = torch.full_like(self.bscales, 99.0)
        for b in range(self.nb):
            L, n = int(self.lens[b]), 1 if new is None else int(new[b])
            if n == 0:
                continue
            for lb in range((L - n) // 16, -(-L // 16)):
                blk = int(self.tables[b, lb])
                k = self.kx[blk, :, :min(16, L - lb * 16)].transpose(0, 1)
                wb, ws = bounds_of(k)
                want_b[blk], want_s[blk] = wb, ws.float()
        assert torch.equal(self.bounds, want_b)
        assert torch.equal(self.bscales, want_s)

    def exact_bounds(self):
        """Every branch's bounds, from the definition."""
        for b in range(self.nb):
            L = int(self.lens[b])
            for lb in range(-(-L // 16)):
                blk = int(self.tables[b, lb])
                wb, ws = bounds_of(
                    self.kx[blk, :, :min(16, L - lb * 16)].transpose(0, 1))
                self.bounds[blk], self.bscales[blk] = wb, ws.float()

    def select(self, n_sel, first, last, null_sel=False):
        n = self.nb * self.Hkv
        sel = torch.full((self.nb, self.Hkv, n_sel), 77, dtype=torch.int32,
                         device="cuda")
        st = torch.full((n, n_sel), 77, dtype=torch.int32, device="cuda")
        sl = torch.full((n,), 77, dtype=torch.int32, device="cuda")
        ws = torch.full((B.paged_select_blocks_workspace_size(
            self.nb, self.mb, self.Hkv),), 0xA5, dtype=torch.uint8, device="cuda")
        B.paged_select_blocks(self.q, self.bounds, self.bscales, self.blocks,
                              self.dt, self.dl, self.nb, self.mb, self.Hq, self.Hkv,
                              self.d, n_sel, first, last, None if null_sel else sel,
                              st, sl, ws)
        assert B.kv_check_device_status(ws) == (0, 0)
        return sel, st, sl

    def want(self, n_sel, first, last):
        G = self.Hq // self.Hkv
        sel = torch.full((self.nb, self.Hkv, n_sel), -1, dtype=torch.int32)
        for b in range(self.nb):
            nblk = -(-int(self.lens[b]) // 16)
            ids = torch.from_numpy(self.tables[b, :nblk].astype(np.int64)).cuda()
            for h in range(self.Hkv):
                if nblk <= n_sel:
                    sel[b, h, :nblk] = torch.arange(nblk)
                    continue
                q = self.q[b, h * G:(h + 1) * G].double()
                odd = ~q.isfinite().all(-1)
                q = torch.where(odd[:, None], 0.0, q)
                p = pow2(exponent(q.abs().amax(-1)))
                n = torch.round(q / p[:, None]).clamp(-127, 127)
                p = torch.where(odd, 0.0, p)
                bd, sc = self.bounds[ids, h].double(), self.bscales[ids, h].double()
                x = torch.maximum(n[:, None] * bd[:, 0], n[:, None] * bd[:, 1])
                x = (x.sum(-1) * p[:, None]).amax(0)
                x = torch.where(sc.isinf(), math.inf, x * sc).cpu()
                always = list(range(first)) + list(range(nblk - last, nblk))
                rest = [j for j in range(first, nblk - last)]
                rest.sort(key=lambda j: (-float(x[j]), j))
                pick = sorted(always + rest[:n_sel - first - last])
                sel[b, h] = torch.tensor(pick, dtype=torch.int32)
        return sel.cuda()

    def check_select(self, n_sel, first, last):
        sel, st, sl = self.select(n_sel, first, last)
        assert torch.equal(sel, self.want(n_sel, first, last))
        for b in range(self.nb):
            nblk = -(-int(self.lens[b]) // 16)
            n = min(nblk, n_sel)
            for h in range(self.Hkv):
                at = sel[b, h, :n].long().cpu()
                phys = torch.from_numpy(self.tables[b])[at].int() * self.Hkv + h
                assert torch.equal(st[b * self.Hkv + h, :n].cpu(), phys)
                assert (st[b * self.Hkv + h, n:] == -1).all()
                assert int(sl[b * self.Hkv + h]) == \
                    16 * n - (16 * nblk - int(self.lens[b]))
        return sel, st, sl

    def attend(self, n_sel, sel, st, sl, sms=152):
        flags = B.KV_PLAN_KV_E4M3 if self.kv == "e4m3" else 0
        plan, info = B.paged_selected_plan(self.nb, self.Hq, self.Hkv, self.d,
                                           self.mb, self.lens, n_sel, sms, flags)
        ws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(self.q)
        tail = (self.blocks, st, sl, self.nb, self.Hq, self.Hkv, self.d, n_sel,
                self.d ** -0.5, out, torch.from_numpy(plan).cuda(), info, ws,
                ws.numel())
        if self.kv == "bf16":
            B.paged_selected_attn(self.q, self.k, self.v, *tail)
        else:
            B.paged_selected_attn_e4m3(self.q, self.k, self.v, self.scales, *tail)
        assert B.kv_check_device_status(ws) == (0, 0)
        G = self.Hq // self.Hkv
        for b in range(self.nb):
            L = int(self.lens[b])
            for h in range(self.Hkv):
                at = sel[b, h][sel[b, h] >= 0].long()
                tok = (at[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
                tok = tok[tok < L]
                k, v = (R.rows(x, self.tables[b], L, h)[tok]
                        for x in (self.kx, self.vx))
                want, tol = R.attend(self.q[b, h * G:(h + 1) * G], k, v,
                                     self.d ** -0.5,
                                     torch.full((G,), len(tok), device="cuda"))
                err = (out[b, h * G:(h + 1) * G].double() - want).abs()
                assert (err <= tol).all()
        return out, info


LENS = [1, 15, 16, 17, 33, 160, 161, 700, 15999]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_bounds_of_steps(Hkv, d, kv):
    t = Tree(Hkv, Hkv, d, LENS, kv)
    t.update()
    t.check_bounds()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 64])
def test_bounds_of_chunks(d, kv):
    """Runs that start and end inside blocks, branches without new tokens, one
    token, whole branches."""
    t = Tree(2, 2, d, [40, 16, 5, 700, 33, 64, 1, 300, 18], kv)
    new = [7, 16, 0, 700, 1, 48, 1, 131, 2]
    t.update(new)
    t.check_bounds(new)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 64])
def test_bounds_of_long_prompts(d, kv):
    """More tiles than warps, of kv-heads that do not come in fours."""
    t = Tree(6, 6, d, [30001, 23, 25000], kv)
    new = [29990, 9, 25000]
    t.update(new)
    t.check_bounds(new)


def test_bounds_of_many_short_runs():
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 90, 300)
    new = np.minimum(lens, rng.integers(0, 6, 300))
    t = Tree(1, 1, 128, lens, seed=3)
    t.update(new)
    t.check_bounds(new)


@pytest.mark.parametrize("d", [128, 64])
def test_bounds_at_the_range_ends(d):
    """Zeros, values at the border of an exponent, tiny and huge ones, one sign."""
    t = Tree(2, 2, d, [16 * 9 + 3])
    vals = [0.0, 127.0, 128.0, -127.5, 2.0 ** -70, 2.0 ** -133, 3e38, 2.0 ** 46,
            -1.0, 0.3]
    for lb, x in enumerate(vals):
        blk = int(t.tables[0, lb])
        if lb == 9:
            t.k[blk].normal_(2.0, 0.1)     # one sign
        else:
            t.k[blk] = 0
            t.k[blk, 0, 2 if lb == 9 else 5 % 16, 11] = x
            t.k[blk, 1] = x
        t.kx[blk] = t.k[blk].double()
    t.update([t.lens[0]])
    t.check_bounds([t.lens[0]])


@pytest.mark.parametrize("x", ["nan", "inf", "-inf"])
def test_bounds_of_keys_that_are_not_finite(x):
    t = Tree(4, 2, 128, [16 * 40])
    blk = int(t.tables[0, 17])
    t.k[blk, 1, 3, 100] = float(x)
    t.kx[blk, 1, 3, 100] = float(x)
    # Behind the end of a branch it counts for nothing.
    u = Tree(2, 2, 128, [16 * 3 + 5])
    last = int(u.tables[0, 3])
    u.k[last, :, 5:] = float(x)
    for y in (t, u):
        y.update([y.lens[0]])
        y.check_bounds([y.lens[0]])
    sel, _, _ = t.check_select(6, 1, 1)
    assert 17 in sel[0, 1].tolist()


def test_bad_blocks_and_lengths_of_bounds_are_reported():
    t = Tree(2, 2, 128, [40, 50])
    t.dt[1, 3] = t.blocks + 9
    with pytest.raises(AssertionError):
        t.update()
    t.dt[1, 3] = int(t.tables[1, 3])
    t.update()
    t.check_bounds()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (8, 8, 64), (14, 2, 128),
                                      (16, 1, 64), (34, 2, 128), (128, 1, 128)])
def test_selected_steps(Hq, Hkv, d, kv):
    t = Tree(Hq, Hkv, d, [1, 200, 2000, 4097, 16 * 24, 16 * 24 + 1, 9000], kv)
    t.exact_bounds()
    t.attend(24, *t.check_select(24, 2, 3))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (3, 1, 64), (40, 2, 128),
                                      (17, 1, 64)])
def test_plans_that_cut_and_that_do_not(Hq, Hkv, d, kv):
    """Whole branches write their results themselves, a CTA or (up to 16 blocks) a warp
    each; halves and more pieces are merged."""
    for n_sel in (9, 40):
        t = Tree(Hq, Hkv, d, [1, 30, 16 * 16, 16 * 17, 3000, 5001, 700], kv, seed=6)
        t.exact_bounds()
        picked = t.check_select(n_sel, 1, 2)
        rows = t.nb * Hkv * -(-Hq // Hkv // 16)
        counts = set()
        for sms in (1, -(-rows * 2 // 7), 152):
            out, info = t.attend(n_sel, *picked, sms=sms)
            counts.add(info.n_row_items == rows)
            again, _ = t.attend(n_sel, *picked, sms=sms)
            assert torch.equal(out, again)
        assert counts == {True, False} or n_sel == 9


@pytest.mark.parametrize("n_sel,first,last", [(1, 0, 1), (2, 1, 1), (2, 0, 2),
                                              (7, 3, 4), (33, 0, 1), (500, 4, 2),
                                              (900, 0, 1)])
def test_budgets(n_sel, first, last):
    t = Tree(8, 2, 128, [13000, 40, 8000, 16], seed=4)
    t.exact_bounds()
    t.attend(n_sel, *t.check_select(n_sel, first, last))


def test_ties_go_to_the_lowest_block():
    """Bounds that repeat every few blocks, and zero queries."""
    t = Tree(4, 2, 64, [16 * 700, 16 * 333 + 1], seed=5)
    t.exact_bounds()
    for b in range(2):
        ids = t.tables[b][t.tables[b] >= 0]
        for j, blk in enumerate(ids):
            t.bounds[int(blk)] = t.bounds[int(ids[j % 5])]
            t.bscales[int(blk)] = t.bscales[int(ids[j % 5])]
    t.check_select(50, 1, 2)
    t.q.zero_()
    t.check_select(50, 1, 2)
    t.q[:, 1] = float("nan")
    t.q[:, 2] = float("inf")
    t.check_select(50, 1, 2)


def test_queries_of_many_sizes():
    t = Tree(4, 2, 128, [16 * 300 + 7], seed=6)
    t.exact_bounds()
    for gain in (1e-30, 1e-12, 1.0, 1e9, 1e30):
        t.q = (torch.randn(1, 4, 128, generator=t.g, device="cuda") * gain).bfloat16()
        t.check_select(20, 0, 1)


def test_negative_scores():
    """Keys opposite to the queries: every bound below zero."""
    t = Tree(2, 1, 128, [16 * 200], seed=7)
    u = torch.randn(128, device="cuda").sign()
    t.k[:] = (-u * (1 + torch.rand(t.k.shape, device="cuda"))).bfloat16()
    t.kx[:] = t.k.double()
    t.q[:] = u.bfloat16()
    t.update([16 * 200])
    t.check_select(12, 0, 1)


def test_a_long_branch():
    t = Tree(8, 1, 128, [16 * 20000 + 3], seed=8)
    t.update([int(t.lens[0])])
    t.check_select(128, 1, 4)


def test_no_logical_list_and_reuse_by_another_layer():
    t = Tree(8, 2, 128, [3000, 500], seed=9)
    t.exact_bounds()
    sel, st, sl = t.select(16, 1, 1)
    _, st2, sl2 = t.select(16, 1, 1, null_sel=True)
    assert torch.equal(st, st2) and torch.equal(sl, sl2)
    t.k, t.v, _, t.kx, t.vx = R.pool(t.blocks, 2, 128, t.g)
    t.attend(16, sel, st, sl)


def test_bad_tables_are_reported():
    t = Tree(8, 2, 128, [3000, 500], seed=10)
    t.exact_bounds()
    t.dt[0, 30] = -7
    with pytest.raises(AssertionError):
        t.select(16, 1, 1)
    t.dt[0, 30] = int(t.tables[0, 30])
    t.check_select(16, 1, 1)


def test_captured_step():
    """Bounds, selection and attention of a decode step in one graph, replayed for
    other keys and queries."""
    t = Tree(8, 2, 128, [2000, 333, 4096], seed=11)
    t.exact_bounds()
    n = t.nb * t.Hkv
    sel = torch.zeros(t.nb, 2, 16, dtype=torch.int32, device="cuda")
    st = torch.zeros(n, 16, dtype=torch.int32, device="cuda")
    sl = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.paged_select_blocks_workspace_size(t.nb, t.mb, 2),
                     dtype=torch.uint8, device="cuda")
    plan, info = B.paged_selected_plan(t.nb, 8, 2, 128, t.mb, t.lens, 16)
    dplan = torch.from_numpy(plan).cuda()
    aws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(t.q)

    def step():
        B.paged_key_bounds(t.k, t.blocks, t.dt, t.dl, None, t.nb, t.nb, t.mb, 2, 128,
                           t.bounds, t.bscales, t.status)
        B.paged_select_blocks(t.q, t.bounds, t.bscales, t.blocks, t.dt, t.dl, t.nb,
                              t.mb, 8, 2, 128, 16, 1, 2, sel, st, sl, ws)
        B.paged_selected_attn(t.q, t.k, t.v, t.blocks, st, sl, t.nb, 8, 2, 128, 16,
                              128 ** -0.5, out, dplan, info, aws, aws.numel())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    t.q.normal_()
    for b in range(t.nb):          # the newest token's key
        blk = int(t.tables[b, (t.lens[b] - 1) // 16])
        x = torch.randn(2, 128, device="cuda").bfloat16()
        t.k[blk, :, (t.lens[b] - 1) % 16] = x
        t.kx[blk, :, (t.lens[b] - 1) % 16] = x.double()
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    t.exact_bounds()
    assert torch.equal(sel, t.want(16, 1, 2))
    t.attend(16, sel, st, sl)
    step()
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_growing_branches_through_the_pool():
    """Prompt, forks inside a block, decode steps with reserved slots: bounds kept up
    to date step by step equal those of the whole branches."""
    Hkv, d, nblk = 2, 64, 64
    k = torch.zeros(1, nblk, Hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    pool = B.kv_pool_create(nblk, 1, Hkv, d, k, v)
    bounds = torch.zeros(nblk, Hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.zeros(nblk, Hkv, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)

    def append(ids, counts):
        n = sum(counts)
        kn, vn = (torch.randn(1, n, Hkv, d, generator=g, device="cuda").bfloat16()
                  for _ in "kv")
        B.kv_append_batch(pool, ids, counts, kn, vn)
        mb = B.kv_batch_max_blocks(pool, ids)
        tables, lens, _ = B.kv_build_batch(pool, ids, mb)
        off = None
        if any(c != 1 for c in counts):
            off = torch.from_numpy(
                np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        B.paged_key_bounds(k[0], nblk, torch.from_numpy(tables).cuda(),
                           torch.from_numpy(lens).cuda(), off, n, len(ids), mb, Hkv,
                           d, bounds, bsc, status)
        return tables, lens

    root = B.kv_branch_create(pool)
    append([root], [75])
    kids = list(B.kv_fork_branches(pool, root, 3))
    for step in range(9):
        tables, lens = append(kids, [1, 1, 1] if step % 3 else [5, 1, 17])
    assert B.kv_check_device_status(status) == (0, 0)
    kx = k[0].double()
    for b in range(3):
        for lb in range(-(-int(lens[b]) // 16)):
            blk = int(tables[b, lb])
            wb, ws = bounds_of(kx[blk, :, :min(16, int(lens[b]) - lb * 16)]
                               .transpose(0, 1))
            assert torch.equal(bounds[blk], wb) and \
                torch.equal(bsc[blk], ws.float())
    B.kv_pool_destroy(pool)
