"""Chunk attention over bf16 and e4m3 pools against the formula in 64 bits."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _chunk_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


class Step:
    """A step over branches of (cached before, new) tokens, `shared` blocks of them
    the same; slots past a branch's length hold NaN."""

    def __init__(self, Hq, Hkv, d, lens, kv="bf16", shared=0, seed=1, sms=0,
                 gain=1.0, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.kv = Hq, Hkv, d, kv
        self.new = np.array([n for _, n in lens], np.int32)
        self.lens = np.array([c + n for c, n in lens], np.int32)
        self.nb, self.total = len(lens), int(self.new.sum())
        nblk = -(-self.lens // 16)
        n_blocks = int(np.maximum(nblk - shared, 0).sum()) + shared + spare
        order = rng.permutation(n_blocks)
        self.tables = np.full((self.nb, max(1, int(nblk.max()))), -1, np.int32)
        at = shared
        for b in range(self.nb):
            k = int(nblk[b])
            self.tables[b, :min(k, shared)] = order[:min(k, shared)]
            if k > shared:
                self.tables[b, shared:k] = order[at:at + k - shared]
                at += k - shared
        self.blocks = n_blocks
        self.k, self.v, self.scales, self.kx, self.vx = R.pool(
            n_blocks, Hkv, d, g, kv)
        self._poison(order[at:], nblk)
        self.q = (torch.randn(self.total, Hq, d, generator=g, device="cuda") *
                  gain).bfloat16()
        self.scale = 1.0 / math.sqrt(d)
        self.plan_sms = sms
        self.plan()

    def _poison(self, free, nblk):
        tails = [(int(self.tables[b, nblk[b] - 1]), int(self.lens[b]) % 16)
                 for b in range(self.nb) if self.lens[b] % 16]
        for blk, t in [(int(f), 0) for f in free] + tails:
            if self.kv == "bf16":
                self.k[blk, :, t:] = float("nan")
                self.v[blk, :, t:] = float("nan")
            else:
                self.v[blk].view(self.Hkv, self.d, 16)[:, :, t:] = 0x7f
                self.k[blk].view(self.Hkv, 16, self.d)[:, t:] = 0x7f

    def plan(self):
        flags = B.KV_PLAN_KV_E4M3 if self.kv == "e4m3" else 0
        plan, self.info = B.paged_chunk_plan(
            self.nb, self.Hq, self.Hkv, self.d, self.blocks, self.tables, self.lens,
            self.new, self.plan_sms, flags)
        self.dplan = torch.from_numpy(plan).cuda()
        self.ws = torch.empty(self.info.workspace_bytes, dtype=torch.uint8,
                              device="cuda").fill_(0xA5)

    def call(self, q, out, stream=None):
        a = (self.blocks, self.total, self.nb, self.Hq, self.Hkv, self.d, self.scale,
             out, self.dplan, self.info, self.ws, self.ws.numel())
        if self.kv == "bf16":
            B.paged_chunk_attn(q, self.k, self.v, *a, stream=stream)
        else:
            B.paged_chunk_attn_e4m3(q, self.k, self.v, self.scales, *a,
                                    stream=stream)

    def run(self):
        # Rows behind the last query stay as they were.
        out = torch.full((self.total + 5, self.Hq, self.d), 7.0,
                         dtype=torch.bfloat16, device="cuda")
        self.call(self.q, out)
        assert B.kv_check_device_status(self.ws) == (0, 0)
        assert (out[self.total:] == 7.0).all()
        return out[:self.total]

    def check(self, out, heads=None):
        row = 0
        G = self.Hq // self.Hkv
        for b in range(self.nb):
            n, L = int(self.new[b]), int(self.lens[b])
            pos = torch.arange(L - n, L, device="cuda")
            for h in heads if heads is not None else range(self.Hq):
                k, v = (R.rows(x, self.tables[b], L, h // G)
                        for x in (self.kx, self.vx))
                want, tol = R.attend(self.q[row:row + n, h], k, v, self.scale, pos)
                err = (out[row:row + n, h].double() - want).abs()
                bad = ~(err <= tol)
                assert not bad.any(), \
                    f"branch {b} head {h}: {int(bad.sum())} values, worst " \
                    f"{float((err / tol).nan_to_num(1e9).max()):.3g} of the bound"
            row += n


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (2, 2), (10, 2), (7, 1), (16, 1),
                                    (33, 1), (128, 1)])
def test_heads(Hq, Hkv, d, kv):
    s = Step(Hq, Hkv, d, [(0, 1), (37, 70), (129, 13), (300, 1)], kv)
    s.check(s.run())


# (cached before, new) around blocks, key tiles of 128 and row tiles.
EDGES = [(0, 1), (0, 15), (0, 16), (0, 17), (1, 1), (15, 1), (16, 1), (127, 1),
         (128, 1), (126, 2), (127, 130), (128, 128), (0, 255), (0, 256), (0, 257),
         (255, 1), (256, 2), (511, 33), (1000, 31), (1, 32), (3, 64)]


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_edge_lengths(G, kv, d):
    s = Step(2 * G, 2, d, EDGES, kv, seed=3)
    s.check(s.run())


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("lens", [[(0, 900)], [(5000, 5)], [(0, 5000)],
                                  [(20000, 3), (0, 1), (777, 300)]])
def test_long(lens, d):
    s = Step(8, 2, d, lens, seed=4)
    s.check(s.run(), heads=[0, 3, 7])


@pytest.mark.parametrize("sms", [2, 16, 152, 2000])
def test_cuts(sms):
    """The same step with key ranges cut for more or fewer SMs."""
    s = Step(8, 2, 128, [(3000, 5), (700, 40), (0, 1), (5000, 1)], seed=5, sms=sms)
    assert (s.info.partial_rows > 0) == (sms > 2)
    s.check(s.run())


def test_branch_without_new_tokens_and_shared_blocks():
    s = Step(16, 2, 128, [(160, 0), (160, 33), (200, 7), (0, 0), (160, 160)],
             shared=10, seed=6)
    s.check(s.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_peaked(kv):
    """Scores that rise with the position, so that maxima move from tile to tile."""
    s = Step(4, 1, 128, [(0, 700), (500, 3)], kv, seed=7, gain=6.0)
    s.check(s.run())


def test_rising_scores():
    s = Step(4, 1, 128, [(0, 640), (900, 20)], seed=8)
    # Keys along one direction, longer and longer.
    u = torch.randn(128, device="cuda").sign()
    for b in range(2):
        for i, blk in enumerate(s.tables[b]):
            if blk < 0:
                continue
            x = (u * (0.02 * (16 * i))).bfloat16()
            s.k[int(blk)] = x
            s.kx[int(blk)] = x.double()
    s.q[:] = u.bfloat16()
    s.check(s.run())


def test_strided_queries():
    """Queries as a slice of a fused projection."""
    s = Step(8, 2, 128, [(10, 50), (300, 9)], seed=9)
    row = torch.randn(s.total, (8 + 4) * 128, device="cuda").bfloat16()
    row[:, :1024] = s.q.flatten(1)
    out = torch.empty_like(s.q)
    s.call(row[:, :1024].unflatten(1, (8, 128)), out)
    want = s.run()
    assert torch.equal(out, want)


def test_same_bits_every_time():
    s = Step(16, 2, 128, [(2000, 33), (100, 500), (4000, 1)], seed=10)
    want = s.run()
    for _ in range(5):
        assert torch.equal(s.run(), want)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("sms", [152, 2])
def test_values_that_are_not_finite(what, bad, kv, sms):
    """A key or value that is not finite reaches only the queries that see it."""
    if kv == "e4m3" and bad != "nan":
        pytest.skip("e4m3 has no infinities")
    d = 128
    for d, lens, t_bad in [(128, [(0, 300)], 150), (128, [(1000, 40)], 1020),
                           (64, [(0, 300)], 299), (128, [(0, 40)], 0),
                           (64, [(1000, 40)], 1003)]:
        s = Step(8, 1, d, lens, kv, seed=11, sms=sms)
        want = s.run().clone()
        blk, t = int(s.tables[0, t_bad // 16]), t_bad % 16
        c = 77 % d
        if kv == "bf16":
            (s.k if what == "k" else s.v)[blk, 0, t, c] = float(bad)
        elif what == "v":
            s.v[blk].view(1, d, 16)[0, c, t] = 0x7f
        else:
            at = t * d + ((((c >> 4) ^ (t & 7)) << 4) + (c & 15) if d == 128 else c)
            s.k[blk, 0, at] = 0x7f
        out = s.run()
        pos = torch.arange(lens[0][0], lens[0][0] + lens[0][1], device="cuda")
        sees = pos >= t_bad
        # (A key of -inf under a positive query only takes its token's weight.)
        assert torch.equal(out[~sees], want[~sees])
        if what == "v":
            col = torch.arange(d, device="cuda") == c
            assert not out[sees][:, :, col].isfinite().any()
            rest = out[sees][:, :, ~col]
            assert torch.equal(rest, want[sees][:, :, ~col])
            if bad != "nan":
                assert (out[sees][:, :, col].float() == float(bad)).all()
        elif bad == "nan":
            assert out[sees].isnan().all()


def test_queries_that_are_not_finite_stay_alone():
    s = Step(8, 2, 128, [(100, 60)], seed=12)
    want = s.run().clone()
    s.q[17, 3, 5] = float("nan")
    out = s.run()
    hit = torch.zeros(60, 8, dtype=torch.bool, device="cuda")
    hit[17, 3] = True
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_captured(kv):
    """Captured into a graph and replayed on other queries; another stream."""
    s = Step(8, 2, 128, [(2000, 5), (30, 200)], kv, seed=13)
    out = torch.empty_like(s.q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.call(s.q, out)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call(s.q, out)
    s.q.copy_(torch.randn_like(s.q.float()).bfloat16())
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    s.check(out)
    assert B.kv_check_device_status(s.ws) == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_behind_work_of_other_streams(kv):
    """Queries that another stream makes, late, captured: the first launch starts early,
    but what reads them does not."""
    s = Step(8, 2, 128, [(2000, 5), (30, 200), (0, 1)], kv, seed=18)
    q, out = torch.zeros_like(s.q), torch.empty_like(s.q)
    slow = torch.randn(4096, 4096, device="cuda")
    s.call(s.q, out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want, n = out.clone(), 3
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            with torch.cuda.stream(side):
                torch.mm(slow, slow)
                q.copy_(s.q)
            here.wait_stream(side)
            s.call(q, out)
            q.fill_(0.0)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_layers_with_one_plan():
    s = Step(8, 2, 128, [(200, 30), (0, 17)], seed=14)
    first = s.run().clone()
    k, v, _, kx, vx = R.pool(s.blocks, 2, 128,
                             torch.Generator(device="cuda").manual_seed(99))
    s.check(first)
    s.k, s.v, s.kx, s.vx = k, v, kx, vx
    s.check(s.run())


def test_bad_block_is_reported():
    """A table entry outside the pool in the device's plan: recorded and skipped."""
    s = Step(8, 2, 128, [(200, 30)], seed=15)
    s.dplan[16 + 3] = s.blocks + 5
    s.call(s.q, torch.empty_like(s.q))
    code, detail = B.kv_check_device_status(s.ws)
    assert (code, detail) == (B.KV_ERR_DEVICE, s.blocks + 5)
    assert B.kv_check_device_status(s.ws) == (0, 0)


def test_nothing_to_do():
    s = Step(8, 2, 128, [(200, 0), (3, 0)], seed=16)
    s.call(None, None)
    assert B.kv_check_device_status(s.ws) == (0, 0)


def test_after_rotating_append():
    """A prompt, then a chunk and a draft, through the calls a model makes: slots
    reserved, queries and keys rotated on the way in, then attention."""
    Hq, Hkv, d = 8, 2, 128
    nblk = 64
    k = torch.full((1, nblk, Hkv, 16, d), float("nan"), dtype=torch.bfloat16,
                   device="cuda")
    v = k.clone()
    pool = B.kv_pool_create(nblk, 1, Hkv, d, k, v)
    a = B.kv_branch_create(pool)
    g = torch.Generator(device="cuda").manual_seed(17)
    ang = torch.arange(512)[:, None] * (10000.0 ** (-torch.arange(64) / 64.0))[None]
    rope = torch.stack([ang.cos(), ang.sin()], -1).float().cuda()
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step(ids, counts):
        B.kv_reserve(pool, ids, counts)
        mb = B.kv_batch_max_blocks(pool, ids)
        tables, lens, _ = B.kv_build_batch(pool, ids, mb)
        n = sum(counts)
        q = torch.randn(n, Hq, d, generator=g, device="cuda").bfloat16()
        kn, vn = (torch.randn(n, Hkv, d, generator=g, device="cuda").bfloat16()
                  for _ in "kv")
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        qr = torch.empty_like(q)
        B.paged_rope_append(q, kn, vn, rope, B.KV_ROPE_HALVES, qr, k[0], v[0], nblk,
                            torch.from_numpy(tables).cuda(),
                            torch.from_numpy(lens).cuda(),
                            torch.from_numpy(off).cuda(), n, len(ids), mb, Hq, Hkv,
                            d, status)
        plan, info = B.paged_chunk_plan(len(ids), Hq, Hkv, d, nblk, tables, lens,
                                        counts)
        ws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        B.paged_chunk_attn(qr, k[0], v[0], nblk, n, len(ids), Hq, Hkv, d, d ** -0.5,
                           out, torch.from_numpy(plan).cuda(), info, ws, ws.numel())
        assert B.kv_check_device_status(ws) == (0, 0)
        kx, vx = k[0].double(), v[0].double()
        for i in range(len(ids)):
            at = slice(off[i], off[i + 1])
            L = int(lens[i])
            pos = torch.arange(L - counts[i], L, device="cuda")
            # What was appended is there: values as they were, keys rotated.
            for h in range(Hkv):
                assert torch.equal(R.rows(vx, tables[i], L, h)[pos],
                                   vn[at, h].double())
                c, sn = (rope[pos][..., j].double() for j in (0, 1))
                x, y = kn[at, h, :64].double(), kn[at, h, 64:].double()
                rot = torch.cat([x * c - y * sn, y * c + x * sn], -1)
                mag = torch.cat([(x * c).abs() + (y * sn).abs(),
                                 (y * c).abs() + (x * sn).abs()], -1)
                # Rounded to bf16 once (2^-8), computed in fp32 (2^-22).
                assert ((R.rows(kx, tables[i], L, h)[pos] - rot).abs() <=
                        rot.abs() * 2.0 ** -8 + mag * 2.0 ** -22).all()
            for h in range(Hq):
                want, tol = R.attend(qr[at, h], R.rows(kx, tables[i], L, h // 4),
                                     R.rows(vx, tables[i], L, h // 4), d ** -0.5,
                                     pos)
                assert ((out[at, h].double() - want).abs() <= tol).all()

    step([a], [70])
    kids = B.kv_fork_branches(pool, a, 3)
    step([a] + list(kids), [5, 40, 1, 130])
    step(list(kids), [1, 1, 3])
    B.kv_pool_destroy(pool)
