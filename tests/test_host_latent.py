"""Latent pools, plans of latent steps and prefills, and the refusals of the
rotating appends and the latent entry points: host logic, no GPU."""

import ctypes as C

import numpy as np
import pytest

from paged_kv_cache_attn_gb300 import binding as B
from paged_kv_cache_attn_gb300 import harness as H
from paged_kv_cache_attn_gb300 import workloads as W


# ---- pools -------------------------------------------------------------------

def test_latent_pool_sizes():
    h = B.kv_pool_create(8, 2, 1, 512, kv_dtype=B.KV_DTYPE_LATENT)
    a = B.kv_branch_create(h)
    B.kv_append(h, a, 20)
    assert B.kv_branch_info(h, a)["n_blocks"] == 2
    b = B.kv_fork_branch(h, a)
    assert B.kv_get_block_table(h, b)[0][0] == B.kv_get_block_table(h, a)[0][0]
    B.kv_pool_destroy(h)
    for heads, d in ((2, 512), (1, 128), (1, 576), (1, 0)):
        with pytest.raises(B.KVError) as e:
            B.kv_pool_create(8, 1, heads, d, kv_dtype=B.KV_DTYPE_LATENT)
        assert e.value.code == B.KV_ERR_INVALID_ARG
    with pytest.raises(B.KVError):
        B.kv_pool_create(8, 1, 1, 512)          # 512 is a latent pool's alone
    with pytest.raises(B.KVError):
        B.kv_pool_create(8, 1, 1, 512, 256, 512, kv_dtype=B.KV_DTYPE_LATENT,
                         kv_scales=1024)
    with pytest.raises(B.KVError):
        B.kv_pool_create(8, 1, 1, 128, kv_dtype=3)


# ---- decode plans --------------------------------------------------------------

def read_plan(plan, info, nb):
    n, pairs, merged = info.n_tile_items, info.n_tile_wide_items, info.n_merge_rows
    items = plan[16:16 + 8 * n].reshape(n, 8)
    o = 16 + 8 * n
    ptr = plan[o:o + pairs + 1]
    o += pairs + 1
    few = plan[o:o + info.n_row_warp_items + 1]
    o += info.n_row_warp_items + 1
    branches = plan[o:o + merged]
    o += merged
    cp = plan[o:o + nb + 1]
    ent = plan[o + nb + 1:].reshape(-1, 4)
    assert o + nb + 1 + 4 * cp[-1] == info.plan_ints == len(plan)
    return items, ptr, few, branches, cp, ent


def check_plan(Hq, lens, groups, plan, info, num_sms):
    nb = len(lens)
    items, ptr, few, branches, cp, ent = read_plan(plan, info, nb)
    # The pairs' lists, then the SMs' lists of items of at most 16 rows.
    assert ptr[0] == 0 and ptr[-1] == few[0] and few[-1] == len(items)
    assert (np.diff(ptr) > 0).all() and (np.diff(few) > 0).all()
    assert len(ptr) - 1 <= max(num_sms // 2, 1)
    assert len(few) - 1 <= 2 * max(num_sms // 2, 1)
    assert info.n_row_items == len(items) - few[0]
    assert (items[few[0]:, 3] <= 16).all()
    # A step of few rows alone is the SMs', a large one of both kinds both's.
    small = items[:, 3] <= 16
    if small.all():
        assert few[0] == 0
    if len(few) > 1:
        assert not small[:few[0]].any()
    # Every (row, block) once.
    seen = [np.zeros((Hq, -(-n // 16)), int) for n in lens]
    rows_of = {}                       # partial row -> (branch, head)
    done = set()                       # rows an item finishes itself
    for b0, direct, row0, nrows, lo, hi, prow, masked in items:
        assert 1 <= nrows <= 128 and lo < hi
        for r in range(row0, row0 + nrows):
            b, h = b0 + r // Hq, r % Hq
            seen[b][h, lo:hi] += 1
            if not masked:
                assert hi * 16 <= lens[b]
            else:
                assert b == b0
            if direct:
                assert (b, h) not in done
                done.add((b, h))
            else:
                k = prow + r - row0
                assert k not in rows_of and k < info.partial_rows
                rows_of[k] = (b, h, lo, hi)
    for s in seen:
        assert (s == 1).all()
    # The merge lists name exactly the partial rows of each branch and head.
    listed = {}
    for b in range(nb):
        for e in ent[cp[b]:cp[b + 1]]:
            base, stride, r_lo, r_hi = e
            for h in range(r_lo, r_hi):
                k = base + h - r_lo
                assert k not in listed
                listed[k] = (b, h)
    assert {k: v[:2] for k, v in rows_of.items()} == listed
    assert sorted(branches) == [b for b in range(nb) if cp[b + 1] > cp[b]]
    for b, h in done:
        assert cp[b + 1] == cp[b]
    assert len(rows_of) == info.partial_rows
    return [[sum(2 * -(-(i[5] - i[4]) // 8) + fixed(i[3])
                 for i in items[x[p]:x[p + 1]]) for p in range(len(x) - 1)]
            for x, fixed in ((ptr, lambda r: 4 + r // 32), (few, lambda r: 2))]


@pytest.mark.parametrize("Hq", [1, 3, 16, 64, 128, 129, 300])
@pytest.mark.parametrize("lens", [[1], [16], [17, 1, 128], [5000], [40] * 300,
                                  [128 * k + 1 for k in range(1, 40)]])
@pytest.mark.parametrize("sms", [152, 2, 1, 0])
def test_latent_plan_independent(Hq, lens, sms):
    mb = max(-(-n // 16) for n in lens)
    plan, info = B.paged_decode_plan(len(lens), Hq, 1, 512, mb, lens, [], sms,
                                     B.KV_PLAN_LATENT)
    check_plan(Hq, lens, [], plan, info, sms or 152)
    assert info.flags == B.KV_PLAN_LATENT
    assert info.workspace_bytes >= 256 + info.partial_rows * (512 * 4 + 8)


@pytest.mark.parametrize("name", ["fanout", "wide", "deep_tree", "tiny_tree"])
@pytest.mark.parametrize("Hq", [2, 16, 128])
def test_latent_plan_trees(name, Hq):
    small = {"wide": dict(n_roots=7, root_tokens=700, fan=40, min_suffix=1,
                          max_suffix=400),
             "fanout": dict(n_roots=3, root_tokens=300, fan=20, min_suffix=1,
                            max_suffix=90),
             "deep_tree": dict(root_tokens=300, depth=3, min_seg=5, max_seg=40),
             "tiny_tree": {}}[name]
    w = W.CONFIGS["fanout" if name == "wide" else name](Hq=Hq, Hkv=1, d=512,
                                                         **small)
    c = H.Cache(w, with_data=False, kv_dtype="latent")
    bt = c.batch(num_sms=152)
    assert len(bt.groups) > 0
    check_plan(Hq, [int(x) for x in bt.seq_lens], bt.groups, bt.plan, bt.info, 152)
    both = bt.info.n_tile_wide_items > 0 and bt.info.n_row_warp_items > 0
    assert both == (name == "wide" and Hq < 128)
    alone = c.batch(num_sms=152, flags=B.KV_PLAN_IGNORE_GROUPS)
    check_plan(Hq, [int(x) for x in alone.seq_lens], [], alone.plan, alone.info, 152)
    c.close()


def test_latent_plan_balances_long_steps():
    """No pair (or SM) of a long step costs more than a few percent above the
    mean."""
    lens = [32768] * 16
    for Hq, which, lists in ((16, 1, 152), (128, 0, 76)):
        plan, info = B.paged_decode_plan(16, Hq, 1, 512, 2048, lens, [], 152,
                                         B.KV_PLAN_LATENT)
        cost = check_plan(Hq, lens, [], plan, info, 152)
        assert not cost[1 - which]
        assert max(cost[which]) <= 1.06 * sum(cost[which]) / lists


def test_latent_plan_refusals():
    ok = dict(nb=1, Hq=4, Hkv=1, head_dim=512, max_blocks=2, seq_lens=[20],
              groups=[], num_sms=152, flags=B.KV_PLAN_LATENT)
    B.paged_decode_plan(**ok)
    for change in (dict(Hkv=2), dict(head_dim=128), dict(head_dim=576),
                   dict(flags=B.KV_PLAN_LATENT | B.KV_PLAN_KV_E4M3),
                   dict(flags=B.KV_PLAN_LATENT | B.KV_PLAN_NO_TENSOR_CORES),
                   dict(flags=0), dict(seq_lens=[0]), dict(seq_lens=[33]),
                   dict(groups=[[0, 1, 0, 2]]), dict(flags=32)):
        with pytest.raises(B.KVError) as e:
            B.paged_decode_plan(**{**ok, **change})
        assert e.value.code == B.KV_ERR_INVALID_ARG, change


# ---- prefill plans -------------------------------------------------------------

def check_prefill_plan(tables, lens, q_lens, plan, info):
    U, T, S = info.n_row_items, info.n_tile_items, info.partial_rows
    uniq, valid = plan[16:16 + U], plan[16 + U:16 + 2 * U]
    slots = plan[16 + 2 * U:16 + 2 * U + S]
    tiles = plan[16 + 2 * U + S:].reshape(T, 4)
    assert len(set(uniq)) == U and info.n_merge_rows == sum(q_lens)
    row = 0
    want = {}
    for b, (L, n) in enumerate(zip(lens, q_lens)):
        for r in range(0, n, 256):
            want[row + r] = (min(256, n - r), L - n + r, b)
        row += n
    assert sorted(t[0] for t in tiles) == sorted(want)
    full = {}
    for row0, nrows, pos0, off in tiles:
        n, p, b = want[row0]
        assert (nrows, pos0) == (n, p)
        nblk = -(-(pos0 + nrows) // 16)
        assert list(uniq[slots[off:off + nblk]]) == list(tables[b][:nblk])
    for b, (L, n) in enumerate(zip(lens, q_lens)):
        if n:
            for k in range(-(-L // 16)):
                x = int(tables[b][k])
                full[x] = max(full.get(x, 0), min(16, L - 16 * k))
    assert dict(zip(map(int, uniq), map(int, valid))) == full
    ends = [t[1] + t[2] for t in tiles]
    assert ends == sorted(ends, reverse=True)


def test_prefill_plan_shares_blocks():
    tables = np.array([[5, 3, 9, -1], [5, 3, 7, 8], [5, 3, 1, -1], [2, -1, -1, -1]])
    lens, q = [40, 60, 48, 7], [40, 3, 0, 7]
    plan, info = B.paged_latent_prefill_plan(4, 8, 16, tables, lens, q)
    check_prefill_plan(tables, lens, q, plan, info)
    assert info.n_row_items == 6            # the idle branch's block 1 is not there
    assert info.workspace_bytes == 256 + 6 * 8 * 8192


@pytest.mark.parametrize("n", [1, 255, 256, 257, 1000])
def test_prefill_plan_tiles(n):
    L = n + 33
    tables = np.arange(-(-L // 16))[None]
    plan, info = B.paged_latent_prefill_plan(1, 3, 100, tables, [L], [n])
    check_prefill_plan(tables, [L], [n], plan, info)


def test_prefill_plan_refusals():
    ok = dict(nb=2, Hq=4, num_blocks=8, tables=[[0, 1], [2, -1]],
              seq_lens=[20, 3], q_lens=[20, 3])
    B.paged_latent_prefill_plan(**ok)
    for change in (dict(Hq=0), dict(num_blocks=0), dict(num_blocks=1),
                   dict(tables=[[0, 8], [2, -1]]), dict(tables=[[0, -1], [2, -1]]),
                   dict(q_lens=[21, 3]), dict(q_lens=[-1, 3]),
                   dict(seq_lens=[33, 3]), dict(seq_lens=[20, 17]),
                   dict(seq_lens=[20])):
        with pytest.raises(B.KVError) as e:
            B.paged_latent_prefill_plan(**{**ok, **change})
        assert e.value.code == B.KV_ERR_INVALID_ARG, change
    # Entries past a branch's blocks are not looked at.
    B.paged_latent_prefill_plan(2, 4, 8, [[0, 99], [2, -5]], [16, 3], [1, 3])


# ---- refusals of the launching calls (before any CUDA call) ----------------------

P = 1 << 20          # a pointer that no refused call follows


def refuse(fn, args, change, what=None):
    a = dict(args)
    a.update(change)
    st = fn(*a.values())
    assert st == B.KV_ERR_INVALID_ARG, (change, st, B.lib().kv_last_error())
    assert B.lib().kv_last_error() != b""


ROPE = dict(q=P, q_stride=512, k=P, k_stride=256, v=P, v_stride=256, rope=P,
            rope_len=10, rot_dim=64, style=0, q_out=P, qo_stride=512, k_pool=P,
            v_pool=P, num_blocks=4, tables=P, lens=P, off=None, total=2, nb=2,
            max_blocks=2, Hq=4, Hkv=2, d=128, bs=16, ws=P, wsb=256, stream=None)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(rope=None),
    dict(tables=None), dict(lens=None), dict(ws=None), dict(k_pool=None),
    dict(q=P + 8), dict(k=P + 2), dict(rope=P + 4), dict(k_pool=P + 8),
    dict(ws=P + 16), dict(wsb=255), dict(q_stride=508), dict(q_stride=504),
    dict(k_stride=248), dict(k_stride=-256), dict(qo_stride=516), dict(rot_dim=0),
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(style=2),
    dict(rope_len=0), dict(d=96), dict(bs=32), dict(Hkv=0), dict(Hq=-1),
    dict(total=3), dict(total=-1, off=P), dict(nb=0, total=0), dict(max_blocks=0),
    dict(num_blocks=0), dict(num_blocks=1 << 31), dict(total=1 << 28, off=P),
])
def test_rope_append_refusals(change):
    refuse(B.lib().paged_rope_append, ROPE, change)
    e = {}
    for k, v in ROPE.items():
        e[k] = v
        if k == "v_pool":
            e["scales"] = P
    refuse(B.lib().paged_rope_append_e4m3, e, change)


def test_rope_append_e4m3_needs_scales():
    e = {}
    for k, v in ROPE.items():
        e[k] = v
        if k == "v_pool":
            e["scales"] = None
    refuse(B.lib().paged_rope_append_e4m3, e, {})
    refuse(B.lib().paged_rope_append_e4m3, e, dict(scales=P + 8))


LAT = dict(c=P, c_stride=576, r=P, r_stride=576, q=P, q_stride=800, q_head=192,
           rope=P, rope_len=10, style=1, qo=P, qo_stride=2304, qo_head=576,
           c_pool=P, r_pool=P, num_blocks=4, tables=P, lens=P, off=P, total=2,
           nb=1, max_blocks=2, Hq=4, rank=512, rope_dim=64, bs=16, ws=P, wsb=256,
           stream=None)


@pytest.mark.parametrize("change", [
    dict(c=None), dict(r=None), dict(q=None), dict(qo=None), dict(c_pool=None),
    dict(r_pool=None), dict(tables=None), dict(lens=None), dict(ws=None),
    dict(c=P + 8), dict(c_stride=504), dict(c_stride=516), dict(r_stride=60),
    dict(q_head=56), dict(q_head=196), dict(q_stride=632), dict(qo_stride=1784),
    dict(rank=256), dict(rope_dim=32), dict(bs=8), dict(style=-1),
    dict(Hq=0), dict(num_blocks=1 << 28), dict(off=None, total=2, nb=1),
])
def test_latent_append_refusals(change):
    refuse(B.lib().paged_latent_append, LAT, change)


def info_of(**kw):
    i = B.kv_decode_plan_info()
    for k, v in kw.items():
        setattr(i, k, v)
    return C.byref(i)


def decode_args():
    return dict(q=P, c=P, r=P, num_blocks=4, tables=P, lens=P, groups=None, ng=0,
                nb=2, mb=2, Hq=4, rank=512, rope_dim=64, bs=16, scale=0.1, out=P,
                plan=P, info=info_of(plan_ints=100, workspace_bytes=256,
                                     n_tile_items=2, n_tile_wide_items=2,
                                     flags=B.KV_PLAN_LATENT),
                ws=P, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(c=None), dict(r=None), dict(tables=None), dict(lens=None),
    dict(out=None), dict(plan=None), dict(info=None), dict(ws=None),
    dict(q=P + 8), dict(out=P + 2), dict(ws=P + 128), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0),
    dict(ng=1), dict(ng=-1), dict(nb=0), dict(Hq=0), dict(mb=0), dict(bs=32),
    dict(rank=128), dict(rope_dim=0), dict(num_blocks=0), dict(wsb=128),
    dict(info=info_of(workspace_bytes=256, n_tile_items=2, n_tile_wide_items=2)),
    dict(info=info_of(workspace_bytes=512, n_tile_items=2, n_tile_wide_items=2,
                      flags=B.KV_PLAN_LATENT)),
    dict(info=info_of(workspace_bytes=256, n_tile_items=0, n_tile_wide_items=0,
                      flags=B.KV_PLAN_LATENT)),
    dict(info=info_of(workspace_bytes=256, n_tile_items=2, n_tile_wide_items=2,
                      n_merge_rows=3, flags=B.KV_PLAN_LATENT)),
])
def test_latent_decode_refusals(change):
    refuse(B.lib().paged_latent_decode_attn, decode_args(), change)


def prefill_args():
    return dict(q=P, c=P, r=P, num_blocks=4, w=P, total=5, nb=2, Hq=2, rank=512,
                rope_dim=64, head_dim=128, bs=16, scale=0.1, out=P, plan=P,
                info=info_of(plan_ints=50, workspace_bytes=256 + 3 * 2 * 8192,
                             n_row_items=3, n_tile_items=1, n_merge_rows=5,
                             partial_rows=3, flags=32),
                ws=P, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(c=None), dict(r=None), dict(w=None), dict(out=None),
    dict(plan=None), dict(info=None), dict(ws=None), dict(w=P + 8),
    dict(ws=P + 64), dict(total=4), dict(total=-1), dict(nb=0), dict(Hq=0),
    dict(Hq=3), dict(rank=64), dict(rope_dim=128), dict(head_dim=64), dict(bs=1),
    dict(scale=0.0), dict(num_blocks=-1), dict(wsb=1000),
    dict(info=info_of(workspace_bytes=256 + 3 * 2 * 8192, n_row_items=3,
                      n_tile_items=1, n_merge_rows=5, partial_rows=3,
                      flags=B.KV_PLAN_LATENT)),
    dict(info=info_of(workspace_bytes=256, n_row_items=0, n_tile_items=1,
                      n_merge_rows=5, flags=32)),
])
def test_latent_prefill_refusals(change):
    refuse(B.lib().paged_latent_prefill_attn, prefill_args(), change)


def test_other_steps_refuse_latent_plans():
    i = info_of(plan_ints=100, workspace_bytes=256, n_tile_items=1,
                n_tile_wide_items=1, n_merge_rows=1, flags=B.KV_PLAN_LATENT)
    st = B.lib().paged_decode_attn(P, P, P, 4, P, P, None, 0, 1, 2, 4, 1, 128, 16,
                                   0.1, P, P, i, P, 1 << 20, None)
    assert st == B.KV_ERR_INVALID_ARG
    assert b"latent" in B.lib().kv_last_error()


def test_rows_and_tables_of_other_types_are_refused():
    """A 16-bit float that is not bf16, or an integer table, has the right size
    and would be read as something else; a tensor of fewer tokens past its end."""
    torch = pytest.importorskip("torch")
    bf = dict(dtype=torch.bfloat16)
    q, kv = torch.zeros(2, 4, 128, **bf), torch.zeros(2, 1, 128, **bf)
    table = torch.zeros(8, 64, 2)
    c, r, qr = (torch.zeros(2, 512, **bf), torch.zeros(2, 64, **bf),
                torch.zeros(2, 4, 64, **bf))
    t64 = torch.zeros(8, 32, 2)

    def rope(**kw):
        a = dict(q=q, k_new=kv, v_new=kv, rope=table, q_out=q, **{})
        a.update(kw)
        B.paged_rope_append(a["q"], a["k_new"], a["v_new"], a["rope"],
                            B.KV_ROPE_HALVES, a["q_out"], P, P, 4, P, P, None, 2,
                            2, 2, 4, 1, 128, torch.zeros(256, dtype=torch.uint8))

    def latent(**kw):
        a = dict(c=c, r=r, qr=qr, rope=t64)
        a.update(kw)
        B.paged_latent_append(a["c"], a["r"], a["qr"], a["rope"], B.KV_ROPE_PAIRS,
                              a["qr"], P, P, 4, P, P, None, 2, 2, 2, 4,
                              torch.zeros(256, dtype=torch.uint8))

    for call, change in ((rope, dict(q=q.half())), (rope, dict(k_new=kv.half())),
                         (rope, dict(v_new=kv.view(torch.int16))),
                         (rope, dict(q_out=q.half())),
                         (rope, dict(rope=table.int())),
                         (rope, dict(q=q[:1])), (rope, dict(k_new=kv[:1])),
                         (rope, dict(q_out=q[:1])), (latent, dict(r=r[:1])),
                         (latent, dict(qr=qr[:1])),
                         (latent, dict(c=c.half())), (latent, dict(r=r.half())),
                         (latent, dict(qr=qr.half())),
                         (latent, dict(rope=t64.int()))):
        with pytest.raises(B.KVError) as e:
            call(**change)
        assert e.value.code == B.KV_ERR_INVALID_ARG


NO_MEMORY = """
import resource, numpy as np
from paged_kv_cache_attn_gb300 import binding as B
used = int(open("/proc/self/statm").read().split()[0]) * 4096
resource.setrlimit(resource.RLIMIT_AS, (used + (64 << 20), used + (64 << 20)))
try:
    B.paged_latent_prefill_plan(1, 1, (2 ** 31 - 1) // 16, np.zeros((1, 1), np.int32),
                                [5], [5])
except B.KVError as e:
    print("refused", e.code)
"""


def test_prefill_plan_without_host_memory():
    """A plan that finds no memory is an error, not the end of the process."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(B.__file__)))
    r = subprocess.run([sys.executable, "-c", NO_MEMORY], cwd=root,
                       capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["refused", str(B.KV_ERR_OOM)], r.stderr[-2000:]
