"""paged_latent_prefill_attn on the GPU, against attention in 64 bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import _latent_ref as LR  # noqa: E402
import _rope_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402

SCALE = 192 ** -0.5


class Step:
    """nb branches of given lengths over a pool of random latents, NaN past
    every branch's length; the first `shared` tokens (whole blocks) are the
    same physical blocks for all of them."""

    def __init__(self, lens, q_lens, Hq, shared=0, seed=1, gain=1.0):
        self.lens, self.q_lens, self.Hq = lens, q_lens, Hq
        nb = len(lens)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        pre = shared // 16
        nblk = [-(-n // 16) for n in lens]
        self.blocks = pre + sum(n - pre for n in nblk) + 3
        order = np.random.default_rng(seed).permutation(self.blocks)
        self.tables = np.full((nb, max(max(nblk), 1)), -1, np.int32)
        at = pre
        self.c = torch.full((self.blocks, 16, 512), float("nan"), device="cuda",
                            dtype=torch.bfloat16)
        self.r = torch.full((self.blocks, 16, 64), float("nan"), device="cuda",
                            dtype=torch.bfloat16)
        for b in range(nb):
            self.tables[b, :pre] = order[:pre]
            k = nblk[b] - pre
            self.tables[b, pre:nblk[b]] = order[at:at + k]
            at += k
            t = np.arange(lens[b])
            blk = torch.from_numpy(self.tables[b][t // 16].astype(np.int64)).cuda()
            slot = torch.from_numpy(t % 16).cuda()
            new = torch.from_numpy((t >= shared) | (b == 0)).cuda()
            self.c[blk[new], slot[new]] = rn(int(new.sum()), 512).bfloat16()
            self.r[blk[new], slot[new]] = rn(int(new.sum()), 64).bfloat16()
        self.n = sum(q_lens)
        self.q = (rn(self.n, Hq, 192) * gain).bfloat16()
        self.w = (rn(Hq, 256, 512) * 512 ** -0.5).bfloat16()
        self.out = torch.full((self.n + 2, Hq, 128), 3.0, device="cuda",
                              dtype=torch.bfloat16)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        plan, self.info = B.paged_latent_prefill_plan(
            nb, Hq, self.blocks, self.tables, lens, q_lens, sms)
        self.plan = torch.from_numpy(plan).cuda()
        # NaN everywhere: nothing of the workspace is read before it is written.
        self.ws = torch.full((self.info.workspace_bytes,), 255,
                             dtype=torch.uint8, device="cuda")

    def run(self, out=None, stream=None):
        B.paged_latent_prefill_attn(
            self.q, self.c, self.r, self.blocks, self.w, self.n, len(self.lens),
            self.Hq, SCALE, self.out[:self.n] if out is None else out, self.plan,
            self.info, self.ws, self.ws.numel(), stream)

    def check(self, heads=None):
        assert B.kv_check_device_status(self.ws) == (0, 0)
        assert (self.out[self.n:] == 3).all()
        off = 0
        for b, (L, n) in enumerate(zip(self.lens, self.q_lens)):
            if n:
                c = LR.tokens(self.c, self.tables[b], L)
                r = LR.tokens(self.r, self.tables[b], L)
                pos = torch.arange(L - n, L, device="cuda")
                for h in range(self.Hq) if heads is None else heads:
                    ref, bound = LR.prefill(self.q[off:off + n, h], c, r,
                                            self.w[h], SCALE, pos)
                    err = (self.out[off:off + n, h].double() - ref).abs()
                    bad = err > bound
                    assert not bad.any(), (b, h, int(bad.sum()),
                                           float((err / bound).max()))
            off += n


CASES = [
    ([1], [1], 1, 0),
    ([5], [5], 3, 0),
    ([16], [16], 2, 0),
    ([127], [127], 2, 0),
    ([128], [128], 2, 0),
    ([129], [129], 2, 0),
    ([256], [256], 1, 0),
    ([257], [257], 2, 0),
    ([300], [1], 4, 0),
    ([300], [130], 2, 0),
    ([1000], [700], 2, 0),
    ([640, 1, 77, 129], [640, 1, 30, 0], 2, 0),
    ([200, 333, 161, 260], [40, 173, 1, 100], 3, 160),
    ([48, 48, 48], [16, 0, 48], 130, 0),
    ([2049], [2049], 2, 0),
]


@pytest.mark.parametrize("lens,q_lens,Hq,shared", CASES)
def test_latent_prefill(lens, q_lens, Hq, shared):
    s = Step(lens, q_lens, Hq, shared)
    s.run()
    torch.cuda.synchronize()
    s.check()
    again = torch.empty_like(s.out[:s.n])
    s.run(again)
    assert torch.equal(again.view(torch.int16), s.out[:s.n].view(torch.int16))


@pytest.mark.parametrize("gain", [0.0, 5.0, 25.0])
def test_flat_and_peaked_scores(gain):
    s = Step([700], [500], 3, seed=3, gain=gain)
    s.run()
    s.check()


def test_long_prompt():
    s = Step([8192], [8192], 8, seed=5)
    s.run()
    s.check(heads=[0, 7])


def test_tree_of_chunks():
    s = Step([4200, 4397, 4801, 4100], [104, 301, 705, 4], 16, shared=4096, seed=6)
    assert s.info.n_row_items == 256 + 7 + 19 + 45 + 1
    s.run()
    s.check(heads=[0, 9, 15])


def test_no_queries():
    s = Step([30, 20], [0, 0], 2)
    assert s.n == 0 and s.info.n_tile_items == 0
    q = torch.zeros(1, 2, 192, dtype=torch.bfloat16, device="cuda")
    B.paged_latent_prefill_attn(q, s.c, s.r, s.blocks, s.w, 0, 2, 2, SCALE, s.out,
                                s.plan, s.info, s.ws, s.ws.numel())
    s.check()


def test_graph_and_two_streams():
    a, b = Step([400], [400], 4, seed=7), Step([900], [300], 4, seed=8)
    a.run()
    torch.cuda.synchronize()
    g, s1, s2 = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s1):
        a.run()
    for seed in (1, 2):
        a.q.copy_(Step([400], [400], 4, seed=seed).q)
        a.out[:a.n] = 0
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g.replay()
        b.run(stream=s2)
        torch.cuda.synchronize()
        a.check()
        b.check()


def test_rising_scores_rescale_every_tile():
    """Scores that rise by more than 8 powers of two a key tile move the maximum,
    and O with it, at every one."""
    s = Step([1500], [600], 2, seed=11)
    t = torch.arange(1500, device="cuda")
    blk = torch.from_numpy(s.tables[0][t.cpu().numpy() // 16].astype(np.int64)).cuda()
    s.r[blk, t % 16] = 0
    s.r[blk, t % 16, 0] = (t // 16).bfloat16()
    s.q.zero_()
    s.q[..., 128] = 14.0        # 14 x 192^-0.5 = 1.01 a block, 8.1 a tile
    s.run()
    s.check()


def test_many_ragged_items():
    """Items of one, two and three key tiles in turn on every pair of SMs."""
    lens = [(37 * i) % 331 + 1 for i in range(48)]
    q_lens = [n if i % 3 else (n + 1) // 2 for i, n in enumerate(lens)]
    s = Step(lens, q_lens, 12, seed=12)
    s.run()
    s.check(heads=[0, 5, 11])
    # 132 heads: groups of heads that do not divide them.
    s = Step([900, 70], [900, 70], 132, seed=13)
    s.run()
    s.check(heads=[0, 63, 131])


def test_bad_plan_entries_are_reported():
    """A block, an index or a tile out of range is recorded, and what does not
    depend on it is right."""
    s = Step([100, 300, 40], [100, 60, 40], 2, seed=14)
    s.run()
    s.check()
    good = s.out.clone()
    U, slots = s.info.n_row_items, s.info.partial_rows
    head = s.info.plan_ints - 4 * s.info.n_tile_items - slots - 2 * U
    for at, value in ((head + U - 1, s.blocks),           # a block of branch 2
                      (head + 2 * U + slots - 1, U),      # its index
                      (head + 2 * U + slots - 1, -1)):
        keep = int(s.plan[at])
        s.plan[at] = value
        s.run()
        assert B.kv_check_device_status(s.ws) == (B.KV_ERR_DEVICE, value)
        assert torch.equal(s.out[:160].view(torch.int16), good[:160].view(torch.int16))
        s.plan[at] = keep
    # Tiles are sorted by their keys: the first is branch 1's.
    at = head + 2 * U + slots
    for field, value in ((0, -1), (0, s.n), (1, 0), (1, 257), (2, -5), (3, -1),
                         (3, slots)):
        keep = int(s.plan[at + field])
        s.plan[at + field] = value
        s.out[:] = 3
        s.run()
        assert B.kv_check_device_status(s.ws)[0] == B.KV_ERR_DEVICE
        for lo, hi, same in ((0, 100, True), (100, 160, False), (160, 200, True)):
            x = s.out[lo:hi].view(torch.int16)
            y = (good[lo:hi] if same else torch.full_like(good[lo:hi], 3.0))
            assert torch.equal(x, y.view(torch.int16)), (field, value, lo)
        s.plan[at + field] = keep
    s.run()
    s.check()


def test_repeated_steps():
    """Hundreds of steps without a pause: no wait runs out, the bits stay."""
    s = Step([700, 333, 90], [300, 333, 1], 16, seed=15)
    s.run()
    s.check(heads=[3])
    first = s.out.clone()
    for _ in range(40):
        for _ in range(10):
            s.run()
        assert B.kv_check_device_status(s.ws) == (0, 0)
        assert torch.equal(s.out.view(torch.int16), first.view(torch.int16))


def test_prompt_then_decode():
    """A prompt enters a latent pool, attends, is forked, and the branches
    decode: append, expanded and absorbed attention over one cache.  The absorbed
    result carried through w_uv is the expanded one's."""
    Hq, n, nblk = 16, 300, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    kp = torch.full((1, nblk, 1, 16, 512), float("nan"), device="cuda",
                    dtype=torch.bfloat16)
    vp = torch.full((1, nblk, 1, 16, 64), float("nan"), device="cuda",
                    dtype=torch.bfloat16)
    h = B.kv_pool_create(nblk, 1, 1, 512, kp, vp, kv_dtype=B.KV_DTYPE_LATENT)
    root = B.kv_branch_create(h)
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    tab = R.table(400, 64).cuda()
    w = (torch.randn(Hq, 256, 512, generator=g, device="cuda") * 512 ** -0.5).bfloat16()
    c, r = kp[0, :, 0], vp[0, :, 0]

    def append(ids, q, row, counts):
        lens = [B.kv_branch_info(h, i)["seq_len"] for i in ids]
        tables, sl, groups = B.kv_build_batch(h, ids)
        assert list(sl) == lens
        dt = torch.from_numpy(tables).cuda()
        dl = torch.from_numpy(sl).cuda()
        off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]),
                           dtype=torch.int32, device="cuda")
        B.paged_latent_append(row[:, :512], row[:, 512:], q[..., 128:], tab,
                              B.KV_ROPE_HALVES, q[..., 128:], c, r, nblk, dt, dl,
                              off, len(row), len(ids), tables.shape[1], Hq, status)
        return tables, sl, groups, dt, dl

    def prefill(ids, q, counts, tables, sl):
        plan, info = B.paged_latent_prefill_plan(len(ids), Hq, nblk, tables, sl,
                                                 counts)
        ws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty(len(q), Hq, 128, dtype=torch.bfloat16, device="cuda")
        B.paged_latent_prefill_attn(q, c, r, nblk, w, len(q), len(ids), Hq, SCALE,
                                    out, torch.from_numpy(plan).cuda(), info, ws,
                                    ws.numel())
        assert B.kv_check_device_status(ws) == (0, 0)
        return out

    def check(ids, q, counts, tables, sl, out):
        o = 0
        for b, k in enumerate(counts):
            L = int(sl[b])
            ct, rt = (LR.tokens(x, tables[b], L) for x in (c, r))
            pos = torch.arange(L - k, L, device="cuda")
            for hh in range(Hq):
                ref, bound = LR.prefill(q[o:o + k, hh], ct, rt, w[hh], SCALE, pos)
                assert ((out[o:o + k, hh].double() - ref).abs() <= bound).all()
            o += k

    q, row = rn(n, Hq, 192), rn(n, 576)
    B.kv_reserve(h, [root], [n])
    tables, sl, _, _, _ = append([root], q, row, [n])
    check([root], q, [n], tables, sl, prefill([root], q, [n], tables, sl))
    kids = B.kv_fork_branches(h, root, 3)
    counts = [5, 1, 20]
    q, row = rn(26, Hq, 192), rn(26, 576)
    B.kv_reserve(h, kids, counts)
    tables, sl, _, _, _ = append(kids, q, row, counts)
    check(kids, q, counts, tables, sl, prefill(kids, q, counts, tables, sl))
    # A decode step of the three branches, both forms.
    q, row = rn(3, Hq, 192), rn(3, 576)
    B.kv_reserve(h, kids, [1] * 3)
    tables, sl, groups, dt, dl = append(kids, q, row, [1] * 3)
    exp = prefill(kids, q, [1] * 3, tables, sl)
    qa = torch.cat([torch.einsum("bhd,hdk->bhk", q[..., :128].float(),
                                 w[:, :128].float()), q[..., 128:].float()],
                   -1).bfloat16()
    plan, info = B.paged_decode_plan(3, Hq, 1, 512, tables.shape[1], sl, groups, 0,
                                     B.KV_PLAN_LATENT)
    ws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(3, Hq, 512, dtype=torch.bfloat16, device="cuda")
    dg = torch.from_numpy(np.ascontiguousarray(groups)).cuda()
    B.paged_latent_decode_attn(qa, c, r, nblk, dt, dl, dg, len(groups), 3,
                               tables.shape[1], Hq, SCALE, out,
                               torch.from_numpy(plan).cuda(), info, ws, ws.numel())
    assert B.kv_check_device_status(ws) == (0, 0)
    assert B.kv_check_device_status(status) == (0, 0)
    for b in range(3):
        ct, rt = (LR.tokens(x, tables[b], int(sl[b])) for x in (c, r))
        ref, bound = LR.decode(qa[b], ct, rt, SCALE)
        assert ((out[b].double() - ref).abs() <= bound).all()
    back = torch.einsum("bhk,hdk->bhd", out.float(), w[:, 128:].float())
    # The forms differ by the rounding of the absorbed query and of the latent
    # result: a few bf16 steps of values of unit scale.
    assert (back - exp.float()).abs().max() < 0.05
    B.kv_pool_destroy(h)
