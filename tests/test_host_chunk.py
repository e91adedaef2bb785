"""Plans of chunk attention and the calls it refuses: host logic, no GPU."""

import os
import subprocess
import sys

import numpy as np
import pytest

from paged_kv_cache_attn_gb300 import binding as B

P = 1 << 20          # a pointer that no call here follows


def layout(lens, shared=0, seed=1):
    rng = np.random.default_rng(seed)
    nblk = [-(-n // 16) for n in lens]
    blocks = sum(max(n - shared, 0) for n in nblk) + shared
    order = rng.permutation(max(blocks, 1))
    t = np.full((len(lens), max(1, max(nblk))), -1, np.int32)
    at = shared
    for b, n in enumerate(nblk):
        t[b, :min(n, shared)] = order[:min(n, shared)]
        if n > shared:
            t[b, shared:n] = order[at:at + n - shared]
            at += n - shared
    return t, max(blocks, 1)


def read(plan, info):
    """(distinct blocks, table entries, items, merges) of a chunk plan."""
    u, it, mg = info.n_row_items, info.n_tile_items, info.n_row_warp_items
    slots = info.plan_ints - 16 - u - 8 * it - 4 * mg
    at = np.cumsum([16, u, slots, 8 * it, 4 * mg])
    return (plan[at[0]:at[1]], plan[at[1]:at[2]], plan[at[2]:at[3]].reshape(-1, 8),
            plan[at[3]:at[4]].reshape(-1, 4))


def check_plan(Hq, Hkv, d, cached, new, sms, flags=0, shared=0):
    lens = [c + n for c, n in zip(cached, new)]
    tables, blocks = layout(lens, shared)
    plan, info = B.paged_chunk_plan(len(lens), Hq, Hkv, d, blocks, tables, lens, new,
                                    sms, flags)
    uniq, slots, items, merges = read(plan, info)
    G = Hq // Hkv
    ctok = 128 // G
    assert info.n_merge_rows == sum(new)
    # Items: more than a CTA's tokens first, each kind longest first.
    wide = items[:, 1] > ctok
    n_wide = int(wide.sum())
    assert n_wide == info.n_tile_wide_items and wide[:n_wide].all()
    keys = items[:, 5] - items[:, 4]
    for part in (keys[:n_wide], keys[n_wide:]):
        assert (np.diff(part) <= 0).all()
    assert (keys >= 1).all()
    if len(keys):
        assert keys.max() * 8 == info.chunk_blocks
    # Every query token has each of its key tiles in one item.
    row, seen = 0, {}
    for r0, n, pos0, table, k0, k1, part, _ in items.tolist():
        assert 1 <= n <= 2 * ctok
        for i in range(n):
            seen.setdefault(r0 + i, []).append((k0, k1, pos0 + i, table, part, r0, n))
    at = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        nblk = -(-lens[b] // 16)
        entry = slots[at:at + nblk]
        phys = uniq[entry] if flags else entry
        assert phys.tolist() == tables[b, :nblk].tolist()
        for i in range(n):
            pieces = sorted(seen.pop(row + i))
            pos = lens[b] - n + i
            assert all(p[2] == pos and p[3] == at for p in pieces)
            last = (pieces[0][2] - i + n - 1)          # the branch's last position
            assert pieces[0][0] == 0
            for x, y in zip(pieces, pieces[1:]):
                assert x[1] == y[0]
            tile_end = pos - (row + i - pieces[0][5]) + pieces[0][6] - 1
            assert pieces[-1][1] == tile_end // 128 + 1 and tile_end <= last
            assert (len(pieces) > 1) == all(p[4] >= 0 for p in pieces)
        row += n
        at += nblk
    assert not seen and at == len(slots)
    # Partial rows: each merge's pieces in its own range, none twice.
    rows = np.zeros(info.partial_rows, int)
    by_row = {int(m[0]): m for m in merges}
    assert len(by_row) == len(merges) == info.n_row_warp_items
    for r0, n, _, _, _, _, part, _ in items.tolist():
        if part < 0:
            assert r0 not in by_row
            continue
        m = by_row[r0]
        k, rest = divmod(part - int(m[2]), n * Hq)
        assert rest == 0 and 0 <= k < m[3] and m[1] == n
        rows[part:part + n * Hq] += 1
    assert (rows == 1).all()
    if flags:
        assert len(set(uniq.tolist())) == len(uniq)
    return info


@pytest.mark.parametrize("flags", [0, B.KV_PLAN_KV_E4M3])
@pytest.mark.parametrize("sms", [2, 30, 152, 1000])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (10, 2), (64, 8), (21, 3), (128, 1)])
def test_plans(Hq, Hkv, sms, flags):
    rng = np.random.default_rng(Hq * 1000 + sms)
    for _ in range(4):
        nb = int(rng.integers(1, 9))
        new = rng.integers(0, 400, nb) * (rng.random(nb) < 0.8)
        new[rng.random(nb) < 0.3] = 1
        cached = rng.integers(0, 3000, nb) * (rng.random(nb) < 0.7)
        check_plan(Hq, Hkv, 128, cached.tolist(), new.tolist(), sms, flags)


def test_plans_of_shared_blocks_and_of_nothing():
    info = check_plan(16, 2, 64, [160, 160, 170], [33, 1, 500], 152,
                      B.KV_PLAN_KV_E4M3, shared=10)
    assert info.n_row_items == 10 + 3 + 1 + (-(-670 // 16) - 10)
    info = check_plan(16, 2, 64, [160, 0], [0, 0], 152)
    assert info.n_tile_items == 0 and info.workspace_bytes == 256


def test_a_few_rows_on_long_branches_are_cut():
    info = check_plan(8, 1, 128, [60000], [3], 152)
    assert info.n_row_warp_items == 1 and info.n_tile_items >= 32
    # Work for all SMs without cuts: none.
    info = check_plan(64, 8, 128, [0], [8192], 152)
    assert info.n_row_warp_items == 0


def refused(f, *a, **k):
    with pytest.raises(B.KVError) as e:
        f(*a, **k)
    assert e.value.code == B.KV_ERR_INVALID_ARG
    return str(e.value)


def test_plans_that_are_refused():
    t, n = layout([40, 50])
    ok = dict(nb=2, Hq=8, Hkv=2, head_dim=128, num_blocks=n, tables=t,
              seq_lens=[40, 50], q_lens=[3, 50])
    B.paged_chunk_plan(**ok)
    for bad in (dict(Hq=9), dict(Hkv=0), dict(Hq=0), dict(Hq=258, Hkv=2),
                dict(head_dim=96), dict(num_blocks=0), dict(num_blocks=1 << 40),
                dict(seq_lens=[40, 49]), dict(q_lens=[-1, 5]), dict(q_lens=[41, 5]),
                dict(seq_lens=[40, 65]), dict(flags=B.KV_PLAN_LATENT),
                dict(flags=1 << 20), dict(num_blocks=n - 1)):
        refused(B.paged_chunk_plan, **{**ok, **bad})
    u = t.copy()
    u[0, 1] = -1
    assert "outside the pool" in refused(B.paged_chunk_plan, **{**ok, "tables": u})


class Rows:
    """As much of a tensor as the binding looks at."""

    def __init__(self, *shape, stride=None, ptr=P):
        torch = pytest.importorskip("torch")
        self.t = torch.empty(0, dtype=torch.bfloat16)
        self.shape, self.dtype, self.ptr = shape, torch.bfloat16, ptr
        self.strides = stride or tuple(
            int(np.prod(shape[i + 1:])) for i in range(len(shape)))

    def stride(self, *a):
        return self.strides[a[0]] if a else self.strides

    def data_ptr(self):
        return self.ptr


def test_steps_that_are_refused():
    t, n = layout([40, 50])
    _, info = B.paged_chunk_plan(2, 8, 2, 128, n, t, [40, 50], [3, 50])
    _, info8 = B.paged_chunk_plan(2, 8, 2, 128, n, t, [40, 50], [3, 50],
                                  flags=B.KV_PLAN_KV_E4M3)
    _, dec = B.paged_decode_plan(2, 8, 2, 128, 4, [40, 50],
                                 np.zeros((0, 4), np.int32), 152)
    q = Rows(53, 8, 128)

    def call(kv="bf16", **kw):
        a = dict(q=q, k=P, v=P, blocks=n, total=53, nb=2, Hq=8, Hkv=2, d=128, scale=0.1,
                 out=q, plan=P, info=info if kv == "bf16" else info8, ws=P,
                 ws_bytes=1 << 40, block_size=16, scales=P)
        a.update(kw)
        head = (a["q"], a["k"], a["v"])
        tail = (a["blocks"], a["total"], a["nb"], a["Hq"], a["Hkv"], a["d"], a["scale"],
                a["out"], a["plan"], a["info"], a["ws"], a["ws_bytes"])
        if kv == "bf16":
            return refused(B.paged_chunk_attn, *head, *tail, stream=0,
                           block_size=a["block_size"])
        return refused(B.paged_chunk_attn_e4m3, *head, a["scales"], *tail, stream=0,
                       block_size=a["block_size"])

    for bad in (dict(k=None), dict(v=None), dict(plan=None), dict(ws=None), dict(q=None),
                dict(out=None), dict(nb=0), dict(total=-1), dict(total=52),
                dict(Hq=9, q=Rows(53, 9, 128), out=Rows(53, 9, 128)),
                dict(Hq=16, q=Rows(53, 16, 128), out=Rows(53, 16, 128)),
                dict(d=64, q=Rows(53, 8, 64), out=Rows(53, 8, 64)),
                dict(Hkv=4), dict(block_size=8), dict(blocks=0), dict(k=P + 8),
                dict(ws=P + 16), dict(scale=0.0), dict(scale=float("nan")),
                dict(ws_bytes=0), dict(info=dec), dict(info=info8),
                dict(q=Rows(53, 8, 128, ptr=P + 2)),
                dict(q=Rows(53, 8, 128, stride=(1028, 128, 1))),
                dict(q=Rows(53, 8, 128, stride=(512, 128, 1))),
                dict(q=Rows(53, 8, 128, stride=(1024, 64, 1))),
                dict(out=Rows(53, 8, 128, stride=(2048, 128, 1))),
                dict(q=Rows(40, 8, 128))):
        call(**bad)
    call("e4m3", scales=None)
    call("e4m3", info=info)
    # A decode step with a plan of a chunk.
    refused(B.paged_decode_attn, P, P, P, n, P, P, None, 0, 2, 4, 8, 2, 128, 0.1, P, P,
            info, P, 1 << 40, stream=0)


NO_MEMORY = """
import resource, numpy as np
from paged_kv_cache_attn_gb300 import binding as B
n = 1 << 19
lens = np.full(n, 256, np.int32)
tables = np.zeros((n, 16), np.int32)
used = int(open("/proc/self/statm").read().split()[0]) * 4096
resource.setrlimit(resource.RLIMIT_AS, (used + (16 << 20), used + (16 << 20)))
try:
    B.paged_chunk_plan(n, 8, 1, 128, 1, tables, lens, lens)
except B.KVError as e:
    print("refused", e.code)
"""


def test_plan_without_host_memory():
    root = os.path.dirname(os.path.dirname(os.path.abspath(B.__file__)))
    r = subprocess.run([sys.executable, "-c", NO_MEMORY], cwd=root,
                       capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["refused", str(B.KV_ERR_OOM)], r.stderr[-2000:]
