"""Selected steps' plans, the calls that selection and beams refuse, and the beams'
reordering of a pool's branches against the model: host logic, no GPU."""

import numpy as np
import pytest

from oracle.allocator import PoolModel, OutOfBlocks
from paged_kv_cache_attn_gb300 import binding as B

P = 1 << 20          # a pointer that no call here follows


def refused(f, *a, **k):
    with pytest.raises(B.KVError) as e:
        f(*a, **k)
    assert e.value.code == B.KV_ERR_INVALID_ARG
    return str(e.value)


class Bytes:
    def __init__(self, n, ptr=P):
        self.n, self.ptr = n, ptr

    def numel(self):
        return self.n

    def data_ptr(self):
        return self.ptr


@pytest.mark.parametrize("flags", [0, B.KV_PLAN_KV_E4M3])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (64, 8), (34, 2), (10, 10)])
@pytest.mark.parametrize("n_sel", [1, 16, 128, 500])
def test_selected_plans_cover_the_selection(Hq, Hkv, n_sel, flags):
    lens = [1, 16, 17, 300, 5000, 16 * 128, 16 * 128 + 1, 9999]
    plan, info = B.paged_selected_plan(len(lens), Hq, Hkv, 128, 700, lens, n_sel, 152,
                                       flags)
    G = Hq // Hkv
    assert info.n_merge_rows == len(lens) * Hkv and info.n_tile_items == 0
    items = plan[16:16 + 8 * info.n_row_items].reshape(-1, 8)
    seen = {}
    for b0, g, r0, n, lo, hi, base, masked in items.tolist():
        assert g == 0 and 0 <= r0 and r0 + n <= G and lo < hi
        for r in range(r0, r0 + n):
            seen.setdefault((b0, r), []).append((lo, hi))
    for b, L in enumerate(lens):
        n = min(-(-L // 16), n_sel)
        for h in range(Hkv):
            for r in range(G):
                got = sorted(seen.pop((b * Hkv + h, r)))
                assert got[0][0] == 0 and got[-1][1] == n
                assert all(x[1] == y[0] for x, y in zip(got, got[1:]))
    assert not seen


def test_selected_plans_that_are_refused():
    ok = dict(nb=2, Hq=8, Hkv=2, head_dim=128, max_blocks=10, seq_lens=[40, 160],
              n_sel=4)
    B.paged_selected_plan(**ok)
    for bad in (dict(nb=0, seq_lens=[]), dict(Hq=9), dict(Hq=260), dict(Hkv=0),
                dict(head_dim=32), dict(max_blocks=0), dict(seq_lens=[0, 5]),
                dict(seq_lens=[40, 161]), dict(n_sel=0), dict(block_size=8),
                dict(flags=B.KV_PLAN_IGNORE_GROUPS), dict(flags=B.KV_PLAN_LATENT)):
        refused(B.paged_selected_plan, **{**ok, **bad})


def test_bounds_that_are_refused():
    def call(e4m3=False, **kw):
        a = dict(k=P, n=10, t=P, l=P, off=P, total=5, nb=2, mb=4, Hkv=2, d=128, b=P,
                 s=P, ws=Bytes(256), bs=16, scales=P)
        a.update(kw)
        tail = (a["n"], a["t"], a["l"], a["off"], a["total"], a["nb"], a["mb"],
                a["Hkv"], a["d"], a["b"], a["s"], a["ws"])
        f, head = (B.paged_key_bounds_e4m3, (a["k"], a["scales"])) if e4m3 else \
            (B.paged_key_bounds, (a["k"],))
        return lambda: f(*head, *tail, stream=0, block_size=a["bs"])

    for bad in (dict(k=None), dict(t=None), dict(l=None), dict(b=None), dict(s=None),
                dict(n=0), dict(n=1 << 40), dict(total=-1), dict(off=None), dict(nb=0),
                dict(mb=0), dict(Hkv=0), dict(d=256), dict(bs=32), dict(k=P + 4),
                dict(b=P + 8), dict(ws=Bytes(128)), dict(ws=Bytes(256, P + 16))):
        refused(call(**bad))
    refused(call(True, scales=None))
    call(total=0)()          # nothing to do


def test_selections_that_are_refused():
    need = B.paged_select_blocks_workspace_size(2, 10, 2)
    assert need >= 256 + 2 * 2 * 10 * 4
    refused(B.paged_select_blocks_workspace_size, 0, 10, 2)

    def call(**kw):
        a = dict(q=P, b=P, s=P, n=10, t=P, l=P, nb=2, mb=10, Hq=8, Hkv=2, d=128, sel=4,
                 first=1, last=1, out=P, st=P, sl=P, ws=Bytes(need), bs=16)
        a.update(kw)
        refused(B.paged_select_blocks, a["q"], a["b"], a["s"], a["n"], a["t"], a["l"],
                a["nb"], a["mb"], a["Hq"], a["Hkv"], a["d"], a["sel"], a["first"],
                a["last"], a["out"], a["st"], a["sl"], a["ws"], stream=0,
                block_size=a["bs"])

    for bad in (dict(q=None), dict(b=None), dict(s=None), dict(t=None), dict(l=None),
                dict(st=None), dict(sl=None), dict(n=0), dict(nb=0), dict(nb=70000),
                dict(mb=0), dict(Hq=9), dict(Hq=258), dict(d=100), dict(sel=0),
                dict(first=-1), dict(last=0), dict(first=3, last=2), dict(q=P + 8),
                dict(b=P + 8), dict(st=P + 2), dict(ws=Bytes(need - 1)),
                dict(ws=Bytes(need, P + 64)), dict(bs=8)):
        call(**bad)
    plan, info = B.paged_selected_plan(2, 8, 2, 128, 10, [40, 160], 4)
    for bad in (dict(Hq=9), dict(nb=3), dict(scale=-1.0), dict(ws_bytes=0)):
        a = dict(nb=2, Hq=8, scale=0.1, ws_bytes=1 << 40)
        a.update(bad)
        refused(B.paged_selected_attn, P, P, P, 10, P, P, a["nb"], a["Hq"], 2, 128, 4,
                a["scale"], P, P, info, P, a["ws_bytes"], stream=0)
    refused(B.paged_selected_attn_e4m3, P, P, P, None, 10, P, P, 2, 8, 2, 128, 4, 0.1, P,
            P, info, P, 1 << 40, stream=0)


def test_beam_selections_that_are_refused():
    torch = pytest.importorskip("torch")
    need = B.kv_beam_select_workspace_size(2, 4, 1000, 8)
    x = torch.zeros(8, 1000)

    def call(**kw):
        a = dict(x=x, s=P, g=2, b=4, n=8, o=P, p=P, t=P, ws=Bytes(need))
        a.update(kw)
        refused(B.kv_beam_select, a["x"], a["s"], a["g"], a["b"], a["n"], a["o"],
                a["p"], a["t"], a["ws"], stream=0)

    for bad in (dict(s=None), dict(o=None), dict(p=None), dict(t=None), dict(g=0),
                dict(b=0), dict(n=0), dict(n=129), dict(g=3), dict(x=x.half()),
                dict(x=x.t()), dict(x=x[:, ::2]), dict(ws=Bytes(need - 256)),
                dict(ws=Bytes(need, P + 8)), dict(s=P + 2),
                dict(x=x[:1].expand(8, 1000)), dict(x=torch.zeros(8, 0))):
        call(**bad)
    for bad in ((0, 1, 10, 1), (1, 0, 10, 1), (1, 1025, 10, 1), (70000, 1, 10, 1),
                (1, 1, 0, 1), (1, 1, 10, 0), (1, 1, 10, 129)):
        refused(B.kv_beam_select_workspace_size, *bad)
    # Any vocabulary will do: the pieces of a row are bounded by the beams alone.
    assert B.kv_beam_select_workspace_size(1, 1024, (1 << 31) - 1, 128) < 2 << 20


# ---- reordering of a pool's branches -----------------------------------------------

def reorder(model, ids, parents):
    """kv_beam_reorder's rule on the model, one branch at a time."""
    used, out = set(), []
    B16 = model.block_size
    need = 0
    for p in parents:
        if p >= 0:
            if p in used:
                need += model.nodes[ids[p]].seq_len % B16 != 0
            used.add(p)
    if need > len(model.free):
        raise OutOfBlocks("forks")
    used = set()
    for p in parents:
        if p < 0:
            out.append(-1)
        elif p in used:
            out.append(model.fork(ids[p])[0])
        else:
            used.add(p)
            out.append(ids[p])
    for k, i in enumerate(ids):
        if k not in used:
            model.free_node(i)
    return out


def same(h, model):
    assert B.kv_get_free_stack(h).tolist() == model.free_stack()
    assert B.kv_get_refcounts(h, model.num_blocks).tolist() == model.ref
    for i, n in enumerate(model.nodes):
        info = B.kv_branch_info(h, i)
        assert info["live"] == int(n.live)
        if n.live:
            table, L = B.kv_get_block_table(h, i)
            assert (table.tolist(), L) == (n.table, n.seq_len)
            assert info["depth"] == n.depth and info["parent"] == n.parent
            assert info["n_children"] == len(n.children)


@pytest.mark.parametrize("seed", range(8))
def test_beams_follow_the_model(seed):
    rng = np.random.default_rng(seed)
    blocks = 120
    order = rng.permutation(blocks).astype(np.int32)
    h = B.kv_pool_create(blocks, 1, 1, 64, None, None, order)
    model = PoolModel(blocks, 16, order.tolist())
    ids = [B.kv_branch_create(h)]
    model.create()
    B.kv_append(h, ids[0], 40)
    model.append(ids[0], 40)
    for _ in range(60):
        n = int(rng.integers(1, 9))
        parents = rng.integers(0, len(ids), n)
        parents[rng.random(n) < 0.1] = -1
        if (parents < 0).all():
            parents[0] = 0
        try:
            want = reorder(model, ids, parents.tolist())
        except OutOfBlocks:
            with pytest.raises(B.KVError) as e:
                B.kv_beam_reorder(h, ids, parents)
            assert e.value.code == B.KV_ERR_OOM
            same(h, model)
            break
        got = B.kv_beam_reorder(h, ids, parents)
        assert got == want
        same(h, model)
        ids = [i for i in got if i >= 0]
        counts = rng.integers(0, 4, len(ids)).tolist()
        try:
            for i, c in zip(ids, counts):
                need = -(-(model.nodes[i].seq_len + c) // 16) - len(model.nodes[i].table)
                if need > len(model.free):
                    raise OutOfBlocks("append")
                model.append(i, c)
                B.kv_append(h, i, c)
        except OutOfBlocks:
            break
        same(h, model)
    B.kv_pool_destroy(h)


def test_beams_that_are_refused_change_nothing():
    h = B.kv_pool_create(4, 1, 1, 64)
    model = PoolModel(4, 16)
    ids = []
    for n in (20, 16, 3):
        i = B.kv_branch_create(h)
        model.create()
        if n != 3:
            B.kv_append(h, i, n)
            model.append(i, n)
        ids.append(i)
    dead = B.kv_branch_create(h)
    model.create()
    B.kv_free(h, dead)
    model.free_node(dead)
    for code, a, p in ((B.KV_ERR_INVALID_ARG, [0, 0], [0, 1]),
                       (B.KV_ERR_NOT_FOUND, [0, 9], [0, 1]),
                       (B.KV_ERR_NOT_FOUND, [0, dead], [0, 0]),
                       (B.KV_ERR_INVALID_ARG, [0, 1], [0, 2]),
                       (B.KV_ERR_INVALID_ARG, [0, 1], [0, -2]),
                       (B.KV_ERR_INVALID_ARG, [], [0]),
                       (B.KV_ERR_OOM, [0, 1], [0, 0, 0])):
        with pytest.raises(B.KVError) as e:
            B.kv_beam_reorder(h, a, p)
        assert e.value.code == code
        same(h, model)
    # Forks of whole blocks need none; branches without tokens fork too.
    assert B.kv_beam_reorder(h, [1, 2], [1, 0, 0, 1, -1]) == \
        reorder(model, [1, 2], [1, 0, 0, 1, -1])
    same(h, model)
    # No beams: all of them freed.
    assert B.kv_beam_reorder(h, [0, 1], []) == reorder(model, [0, 1], [])
    assert B.kv_beam_reorder(h, [], []) == []
    same(h, model)
    B.kv_pool_destroy(h)


def test_spilled_branches_go_on_alone():
    """A spilled branch keeps its place in the beams, but is not forked."""
    h = B.kv_pool_create(8, 1, 1, 64)
    B.kv_offload_attach(h, None, None, 8)
    a, b = B.kv_branch_create(h), B.kv_branch_create(h)
    B.kv_append(h, a, 20)
    B.kv_append(h, b, 20)
    B.kv_spill(h, [a])
    refused(B.kv_beam_reorder, h, [a, b], [0, 0])
    assert B.kv_beam_reorder(h, [a, b], [0, 1, 1]) == [a, b, 2]
    assert B.kv_beam_reorder(h, [a, b, 2], [2]) == [2]
    assert len(B.kv_get_host_free(h)) == 8
    B.kv_pool_destroy(h)
