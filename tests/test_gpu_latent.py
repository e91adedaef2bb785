"""paged_latent_decode_attn on the GPU, against attention in 64 bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import _latent_ref as LR  # noqa: E402
import _rope_ref as R  # noqa: E402
from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402
from paged_kv_cache_attn_gb300 import harness as H  # noqa: E402
from paged_kv_cache_attn_gb300 import workloads as W  # noqa: E402


def latent(w):
    w.Hkv, w.d = 1, 512
    return w


def lengths(lens, Hq):
    w = W.Workload("lengths", Hq, 1, 512, 31)
    for i, n in enumerate(lens):
        w.nodes.append(W.NodeSpec(-1, int(n)))
        w.ops += [("create",), ("append", i)]
    w.num_blocks = sum(-(-n // 16) for n in lens) + 3
    return w


CASES = {
    "one_token": lambda: lengths([1], 1),
    "one_token_128": lambda: lengths([1] * 5, 128),
    "block_edges": lambda: lengths([1, 15, 16, 17, 31, 32, 33, 48], 16),
    "tile_edges": lambda: lengths([63, 64, 65, 127, 128, 129, 191, 192, 193,
                                   255, 256, 257], 3),
    "odd_heads": lambda: lengths([300, 77], 130),
    "heads_257": lambda: lengths([143], 257),
    "many_short": lambda: lengths([1 + (7 * i) % 40 for i in range(400)], 16),
    "split": lambda: lengths([5000], 16),
    "split_128": lambda: lengths([4097, 513], 128),
    "tiny_tree": lambda: latent(W.tiny_tree()),
    "fanout": lambda: latent(W.fanout(n_roots=2, root_tokens=256, fan=8,
                                      min_suffix=1, max_suffix=100, Hq=16)),
    # Enough of both kinds of items for the two kernels beside each other.
    "fanout_both": lambda: latent(W.fanout(n_roots=4, root_tokens=300, fan=48,
                                           min_suffix=1, max_suffix=260, Hq=16)),
    "fanout_3tiles": lambda: latent(W.fanout(n_roots=1, root_tokens=777,
                                             fan=40, min_suffix=1,
                                             max_suffix=50, Hq=9)),
    "deep_tree": lambda: latent(W.deep_tree(root_tokens=300, depth=3,
                                            min_seg=5, max_seg=40, Hq=16)),
    "long": lambda: latent(W.long_context(n_indep=3, indep_tokens=1000,
                                          n_roots=2, root_tokens=2048, fan=16,
                                          suffix_tokens=37, Hq=128)),
}


def queries(nb, Hq, seed, gain=0.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randn(nb, Hq, 576, generator=g, device="cuda")
    q[..., :512] *= gain
    return q.bfloat16()


def check(c, bt, q, out, what, rows=None):
    for b in range(bt.nb) if rows is None else rows:
        L = int(bt.seq_lens[b])
        ct = LR.tokens(c.k[0, :, 0], bt.tables[b], L)
        rt = LR.tokens(c.v[0, :, 0], bt.tables[b], L)
        ref, bound = LR.decode(q[b], ct, rt, c.scale)
        err = (out[b].double() - ref).abs()
        bad = err > bound
        assert not bad.any(), (what, b, L, int(bad.sum()), float(err.max()),
                               float((err / bound).max()))


@pytest.mark.parametrize("flags", [0, B.KV_PLAN_IGNORE_GROUPS])
@pytest.mark.parametrize("name", list(CASES))
def test_latent_decode(name, flags):
    """Every row of every branch; slots past the lengths hold NaN."""
    w = CASES[name]()
    c = H.Cache(w, kv_dtype="latent", poison=True)
    bt = c.batch(flags=flags).upload()
    q = queries(bt.nb, w.Hq, 3)
    out = torch.full((bt.nb + 1, w.Hq, 512), 3.0, dtype=torch.bfloat16,
                     device="cuda")
    bt.decode(q, out[:-1])
    torch.cuda.synchronize()
    assert bt.device_status() == (0, 0)
    assert (out[-1] == 3).all()              # rows behind the last branch
    check(c, bt, q, out, name)
    # The same call again gives the same bits.
    again = torch.empty_like(out[:-1])
    bt.decode(q, again)
    assert torch.equal(again.view(torch.int16), out[:-1].view(torch.int16))
    c.close()


@pytest.mark.parametrize("gain", [0.0, 4.0, 30.0])
def test_peaked_and_flat_scores(gain):
    """Scores whose maximum moves from tile to tile (O is rescaled), and equal
    ones (the mean)."""
    w = lengths([1000, 130, 4000], 24)
    c = H.Cache(w, kv_dtype="latent", poison=True)
    bt = c.batch().upload()
    q = queries(bt.nb, w.Hq, 5, gain)
    if gain == 0.0:
        q.zero_()
    out = torch.empty((bt.nb, w.Hq, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, gain)
    c.close()


def test_rising_scores_rescale_every_tile():
    """Token t's score grows with t, so that every tile raises the maximum."""
    w = lengths([2000], 16)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    L = 2000
    t = torch.from_numpy(bt.tables[0].astype(np.int64)).cuda()
    ramp = torch.zeros(len(t) * 16, device="cuda")
    ramp[:L] = torch.arange(L, device="cuda") * 0.25
    c.v[0, :, 0, :, :] = 0
    c.v[0, t, 0, :, 0] = ramp.view(-1, 16).bfloat16()
    q = queries(1, 16, 7)
    q[..., 512:] = 0
    q[..., 512] = 8.0
    out = torch.empty((1, 16, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, "ramp")
    c.close()


@pytest.mark.parametrize("lens,Hq", [([600] * 170, 16), ([2000, 700], 128),
                                     ([333] * 90, 24), ([1500, 40], 1)])
def test_rising_scores_of_whole_branches(lens, Hq):
    """The same where an item has many tiles: long lists, 1 to 128 rows."""
    w = lengths(lens, Hq)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    c.v[0, :, 0, :, :] = 0
    for b, L in enumerate(lens):
        t = torch.from_numpy(bt.tables[b][:-(-L // 16)].astype(np.int64)).cuda()
        ramp = torch.arange(len(t) * 16, device="cuda") * 0.25
        c.v[0, t, 0, :, 0] = ramp.view(-1, 16).bfloat16()
    q = queries(len(lens), Hq, 7)
    q[..., 512:] = 0
    q[..., 512] = 8.0
    out = torch.empty((len(lens), Hq, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, "ramp", rows=range(0, len(lens), 13))
    c.close()


@pytest.mark.parametrize("name", ["fanout_both", "many_short", "split_128", "long"])
def test_repeated_steps(name):
    """Hundreds of steps without a pause: no wait runs out, the bits stay."""
    w = CASES[name]()
    c = H.Cache(w, kv_dtype="latent", poison=True)
    bt = c.batch().upload()
    both = bt.info.n_tile_wide_items > 0 and bt.info.n_row_warp_items > 0
    assert both == (name == "fanout_both")
    q = queries(bt.nb, w.Hq, 11)
    first = torch.empty((bt.nb, w.Hq, 512), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(first)
    bt.decode(q, first)
    assert bt.device_status() == (0, 0)
    for _ in range(40):
        for _ in range(10):
            bt.decode(q, out)
        assert bt.device_status() == (0, 0)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    c.close()


def test_bad_block_ids_of_many_rows():
    w = lengths([100, 300], 48)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    q = queries(2, 48, 2)
    out = torch.empty((2, 48, 512), dtype=torch.bfloat16, device="cuda")
    for bad in (w.num_blocks, -1, 1 << 30):
        bt.dev["tables"][1, 4] = bad
        bt.decode(q, out)
        assert bt.device_status() == (B.KV_ERR_DEVICE, bad)
    bt.dev["tables"][1, 4] = int(bt.tables[1, 4])
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, "after")
    c.close()


@pytest.mark.parametrize("name,Hq", [("independent", 128), ("fanout", 16),
                                     ("deep_tree", 16)])
def test_full_size(name, Hq):
    w = W.CONFIGS[name](Hq=Hq, Hkv=1, d=512)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    q = queries(bt.nb, Hq, 13)
    out = torch.empty((bt.nb, Hq, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, name)
    c.close()


def test_shared_and_private_layouts_agree():
    """The same tokens shared through segments and read per branch."""
    w = CASES["fanout"]()
    c = H.Cache(w, kv_dtype="latent")
    q = queries(len(c.decode_ids), w.Hq, 1)
    outs = []
    for flags in (0, B.KV_PLAN_IGNORE_GROUPS):
        bt = c.batch(flags=flags).upload()
        o = torch.empty((bt.nb, w.Hq, 512), dtype=torch.bfloat16, device="cuda")
        bt.decode(q, o)
        outs.append(o.float())
    assert (outs[0] - outs[1]).abs().max() < 0.05
    c.close()


def test_bad_block_ids_are_reported():
    w = lengths([100, 300], 16)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    q = queries(2, 16, 2)
    out = torch.empty((2, 16, 512), dtype=torch.bfloat16, device="cuda")
    for bad in (w.num_blocks, -1, 1 << 30):
        bt.dev["tables"][1, 4] = bad
        bt.decode(q, out)
        assert bt.device_status() == (B.KV_ERR_DEVICE, bad)
    bt.dev["tables"][1, 4] = int(bt.tables[1, 4])
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, "after")
    c.close()


def test_graphs_and_streams():
    """Captured on a side stream, replayed with new queries; two steps with
    workspaces of their own on two streams at once."""
    w = CASES["fanout"]()
    c = H.Cache(w, kv_dtype="latent")
    b1, b2 = c.batch().upload(), c.batch(flags=B.KV_PLAN_IGNORE_GROUPS).upload()
    q = queries(b1.nb, w.Hq, 1)
    o1 = torch.zeros((b1.nb, w.Hq, 512), dtype=torch.bfloat16, device="cuda")
    o2 = torch.zeros_like(o1)
    b1.decode(q, o1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s1):
        b1.decode(q, o1)
    for seed in (2, 3):
        q.copy_(queries(b1.nb, w.Hq, seed))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g.replay()
        b2.decode(q, o2, stream=s2)
        torch.cuda.synchronize()
        check(c, b1, q, o1, "graph")
        check(c, b2, q, o2, "stream")
    c.close()


def test_layer_loop_append_then_decode():
    """Decode steps as an engine runs them: reserve, then per layer append
    (rotated) and attend, over a forked tree; pools of three layers."""
    w = latent(W.tiny_tree())
    w.num_layers, w.Hq = 3, 16
    c = H.Cache(w, kv_dtype="latent", poison=True)
    ids = c.decode_ids
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tab = R.table(400, 64).cuda()
    for step in range(18):                     # past a block's end
        B.kv_reserve(c.h, ids, [1] * len(ids))
        bt = c.batch().upload()
        for layer in range(3):
            row = torch.randn(bt.nb, 576, generator=g, device="cuda").bfloat16()
            q = queries(bt.nb, w.Hq, 100 * step + layer)
            pre = q.clone()
            bt.append_rotated(q[..., 512:], row[:, :512], row[:, 512:], tab,
                              B.KV_ROPE_PAIRS, q[..., 512:], layer=layer)
            out = torch.empty((bt.nb, w.Hq, 512), dtype=torch.bfloat16,
                              device="cuda")
            bt.decode(q, out, layer=layer)
            assert bt.append_status() == (0, 0)
            assert bt.device_status() == (0, 0)
            pos = torch.from_numpy(bt.seq_lens.astype(np.int64) - 1).cuda()
            y, mag = R.rotate(pre[..., 512:], tab, pos, True)
            assert ((q[..., 512:].double() - y).abs() <= R.bf16_bound(y, mag)).all()
            if step % 5 == 0 or step == 17:
                for b in range(bt.nb):
                    L = int(bt.seq_lens[b])
                    ct = LR.tokens(c.k[layer, :, 0], bt.tables[b], L)
                    rt = LR.tokens(c.v[layer, :, 0], bt.tables[b], L)
                    ref, bound = LR.decode(q[b], ct, rt, c.scale)
                    assert torch.equal(ct[-1], row[b, :512].double())
                    assert ((out[b].double() - ref).abs() <= bound).all()
    c.close()


def test_fork_spill_and_restore_of_a_latent_pool():
    """Copy-on-write and the host tier carry latents and position keys."""
    w = latent(W.tiny_tree())
    w.Hq = 4
    c = H.Cache(w, kv_dtype="latent")
    hk = torch.empty((1, 8, 1, 16, 512), dtype=torch.bfloat16).pin_memory()
    hv = torch.empty((1, 8, 1, 16, 64), dtype=torch.bfloat16).pin_memory()
    B.kv_offload_attach(c.h, hk, hv, 8)
    torch.cuda.synchronize()

    def rows(i):
        t, L = B.kv_get_block_table(c.h, i)
        return (LR.tokens(c.k[0, :, 0], t, L), LR.tokens(c.v[0, :, 0], t, L))

    for i in c.decode_ids:                      # the forks copied the root's tail
        k, v = w.node_kv(0)
        want = torch.from_numpy(k[0, :, 0].view(np.int16)).view(torch.bfloat16)
        assert torch.equal(rows(i)[0][:100].cpu(), want.double())
        want = torch.from_numpy(np.ascontiguousarray(v[0, :, 0, :64]).view(np.int16))
        assert torch.equal(rows(i)[1][:100].cpu(),
                           want.view(torch.bfloat16).double())
    i = c.decode_ids[1]
    before = rows(i)
    assert B.kv_spill(c.h, [i]) > 0
    B.kv_restore(c.h, [i])
    torch.cuda.synchronize()
    after = rows(i)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    c.close()
