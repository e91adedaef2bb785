"""Latent steps at the edges of their plans on the GPU, against attention in 64
bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402
from paged_kv_cache_attn_gb300 import harness as H  # noqa: E402
from paged_kv_cache_attn_gb300 import workloads as W  # noqa: E402
from test_gpu_latent import check, queries  # noqa: E402


def forked(root_tokens, tails, Hq):
    """Branches forked from one root; a tail of 0 tokens ends with the root."""
    w = W.Workload("forked", Hq, 1, 512, 37)
    w.nodes.append(W.NodeSpec(-1, root_tokens))
    w.ops += [("create",), ("append", 0), ("fork", 0, len(tails))]
    for i, n in enumerate(tails):
        w.nodes.append(W.NodeSpec(0, n))
        if n:
            w.ops.append(("append", i + 1))
    w.num_blocks = -(-root_tokens // 16) + sum(-(-n // 16) for n in tails) + 3
    return w


@pytest.mark.parametrize("Hq,root,tails", [
    (48, 32, [8, 8, 0]), (48, 32, [0, 0, 0, 1]), (20, 32, [0] * 6 + [18]),
    (9, 64, [1] + [0] * 14), (9, 64, [0] * 30 + [40] + [0] * 30),
    (96, 640, [0, 0, 6, 0]), (200, 160, [0, 5, 0])])
def test_branches_that_end_with_their_segment(Hq, root, tails):
    w = forked(root, tails, Hq)
    c = H.Cache(w, kv_dtype="latent", poison=True)
    bt = c.batch().upload()
    assert [list(g) for g in bt.groups] == [[0, len(tails), 0, root // 16]]
    q = queries(bt.nb, Hq, 3)
    out = torch.full((bt.nb, Hq, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    assert torch.isfinite(out).all()
    check(c, bt, q, out, "forked")
    c.close()


def test_merge_entries_out_of_place_are_reported():
    """A head without a partial row is recorded and left as it was."""
    w = forked(320, [50, 50, 70], 16)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    q = queries(3, 16, 4)
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    check(c, bt, q, out, "before")
    i = bt.info
    ptr = 16 + 8 * i.n_tile_items + i.n_tile_wide_items + i.n_row_warp_items + 2 + \
        i.n_merge_rows
    cp = bt.plan[ptr:ptr + 4]
    assert cp[2] > cp[1]
    good = out.clone()
    for e in range(cp[1], cp[2]):                 # branch 1: heads 0 to 4 only
        bt.dev["plan"][ptr + 4 + 4 * int(e) + 3] = 5
    out[:] = 3
    bt.decode(q, out)
    assert bt.device_status() == (B.KV_ERR_DEVICE, -2)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert torch.equal(out[1, :5], good[1, :5]) and (out[1, 5:] == 3).all()
    c.close()


def test_prefill_of_no_tokens_does_nothing():
    """Empty tensors have no address; the status is cleared all the same."""
    blocks, Hq = 8, 4
    pools = [torch.zeros(blocks, 16, n, dtype=torch.bfloat16, device="cuda")
             for n in (512, 64)]
    plan, info = B.paged_latent_prefill_plan(2, Hq, blocks, [[0, 1], [2, 3]],
                                             [20, 30], [0, 0])
    plan = torch.from_numpy(plan).cuda()
    ws = torch.full((info.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    w = torch.zeros(Hq, 256, 512, dtype=torch.bfloat16, device="cuda")
    e = dict(dtype=torch.bfloat16, device="cuda")
    B.paged_latent_prefill_attn(torch.empty(0, Hq, 192, **e), *pools, blocks, w, 0,
                                2, Hq, 0.1, torch.empty(0, Hq, 128, **e), plan,
                                info, ws, ws.numel())
    assert B.kv_check_device_status(ws) == (0, 0)


def test_prefill_bits_do_not_depend_on_which_pair_takes_an_item():
    """Hundreds of items of one to nine key tiles, most handed out as pairs of SMs
    come free, so that an item follows others in every run."""
    from test_gpu_latent_prefill import Step
    lens = [260 + (193 * i) % 900 for i in range(60)]
    q_lens = [min(n, 30 + (71 * i) % 400) for i, n in enumerate(lens)]
    s = Step(lens, q_lens, 12, seed=21)
    s.run()
    s.check(heads=[0, 11])
    first = s.out.clone()
    differ = 0
    for _ in range(30):
        for _ in range(5):
            s.run()
        differ += not torch.equal(s.out.view(torch.int16), first.view(torch.int16))
    assert B.kv_check_device_status(s.ws) == (0, 0)
    assert differ == 0


@pytest.mark.parametrize("value", [1 << 20, (1 << 31) - 1, -1, -(1 << 31)])
def test_merge_lists_out_of_range_are_reported(value):
    w = forked(320, [50, 50, 70], 16)
    c = H.Cache(w, kv_dtype="latent")
    bt = c.batch().upload()
    q = queries(3, 16, 4)
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda")
    bt.decode(q, out)
    assert bt.device_status() == (0, 0)
    good = out.clone()
    i = bt.info
    ptr = 16 + 8 * i.n_tile_items + i.n_tile_wide_items + i.n_row_warp_items + 2 + \
        i.n_merge_rows
    bt.dev["plan"][ptr + 2] = value              # branch 1's end, branch 2's start
    out[:] = 3
    bt.decode(q, out)
    code, detail = bt.device_status()
    assert code == B.KV_ERR_DEVICE and detail in (-2, -3)
    assert torch.equal(out[0], good[0])
    assert (out[1:] == 3).all()
    c.close()


@pytest.mark.parametrize("what", ["nan", "inf", "key"])
def test_a_bad_token_reaches_only_the_rows_that_see_it(what):
    """A latent with a NaN or an infinity, or a position key with a NaN: the queries
    before that token get the bits that they have without it, those from it on NaN."""
    from test_gpu_latent_prefill import Step
    s = Step([700, 200, 160], [700, 40, 0], 3, shared=160, seed=22)
    s.run()
    s.check()
    good = s.out.clone()
    for t in (0, 15, 300, 511, 699):
        blk, slot = int(s.tables[0][t // 16]), t % 16
        keep = s.c[blk, slot].clone(), s.r[blk, slot].clone()
        if what == "key":
            s.r[blk, slot, 5] = float("nan")
        else:
            s.c[blk, slot, 77] = float(what)
        s.out[:] = 3
        s.run()
        assert B.kv_check_device_status(s.ws) == (0, 0)
        sees = torch.arange(s.n, device="cuda") >= t
        sees[700:] = t < 160                  # the other branch shares 160 tokens
        got, want = s.out[:s.n], good[:s.n]
        assert torch.equal(got[~sees].view(torch.int16), want[~sees].view(torch.int16))
        assert got[sees].isnan().all()
        s.c[blk, slot], s.r[blk, slot] = keep
    s.run()
    assert torch.equal(s.out.view(torch.int16), good.view(torch.int16))
