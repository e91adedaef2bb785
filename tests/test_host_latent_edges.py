"""Plans of latent steps where few units share branches, and the calls of steps
without new tokens: host logic, no GPU."""

import numpy as np
import pytest

from paged_kv_cache_attn_gb300 import binding as B
from test_host_latent import check_plan


# Branches that end with the shared segment (one unit each) beside branches with
# tails (two), where 128 rows are no whole number of branches: a branch's heads lie
# in two row tiles of the segment.  (Hq, lens, segments.)
STRADDLING = [
    (48, [40, 40, 32], [[0, 3, 0, 2]]),
    (48, [32, 32, 32, 33], [[0, 4, 0, 2]]),
    (20, [32] * 6 + [50], [[0, 7, 0, 2]]),
    (20, [50] + [32] * 19, [[0, 20, 0, 2]]),
    (9, [33] + [32] * 14, [[0, 15, 0, 2]]),
    (9, [32] * 30 + [33] + [32] * 30, [[0, 61, 0, 2]]),
    (96, [64, 64, 70, 64], [[0, 4, 0, 4]]),
    # Two levels: the second segment's branches have two units each.
    (48, [32, 32, 64, 64, 32], [[0, 5, 0, 2], [2, 2, 2, 2]]),
    # Long segments, cut into pieces, one after another.
    (48, [16000] * 5 + [16010] * 3 + [8000] * 4, [[0, 8, 0, 1000], [8, 4, 0, 500]]),
    (200, [8000] * 3, [[0, 3, 0, 500]]),
]


@pytest.mark.parametrize("sms", [152, 4, 1])
@pytest.mark.parametrize("case", range(len(STRADDLING)))
def test_rows_are_finished_or_merged_and_not_both(case, sms):
    """A branch whose heads lie in two items is finished by both or merged."""
    Hq, lens, groups = STRADDLING[case]
    plan, info = B.paged_decode_plan(len(lens), Hq, 1, 512,
                                     max(-(-n // 16) for n in lens), lens, groups,
                                     sms, B.KV_PLAN_LATENT)
    check_plan(Hq, lens, groups, plan, info, sms)


@pytest.mark.parametrize("seed", range(24))
def test_random_segments(seed):
    """Segments one beside another and below one another, some branches ending
    with theirs, in every head count."""
    rng = np.random.default_rng(seed)
    Hq = int(rng.choice([1, 5, 9, 16, 20, 48, 96, 127, 129, 200]))
    lens, groups = [], []
    while len(lens) < 40:
        n, blocks = int(rng.integers(1, 16)), int(rng.integers(1, 200))
        b0 = len(lens)
        end = [blocks] * n
        if n > 1:
            groups.append([b0, n, 0, blocks])
            k = int(rng.integers(0, n))            # the first k: one level more
            if k > 1:
                more = int(rng.integers(1, 30))
                groups.append([b0, k, blocks, more])
                end[:k] = [blocks + more] * k
        lens += [16 * e + int(rng.integers(1, 60)) * int(rng.random() < 0.4)
                 for e in end]
    plan, info = B.paged_decode_plan(len(lens), Hq, 1, 512,
                                     max(-(-n // 16) for n in lens), lens, groups,
                                     152, B.KV_PLAN_LATENT)
    check_plan(Hq, lens, groups, plan, info, 152)


def layout(Hq, lens, groups):
    plan, info = B.paged_decode_plan(len(lens), Hq, 1, 512,
                                     max(-(-n // 16) for n in lens), lens, groups,
                                     152, B.KV_PLAN_LATENT)
    check_plan(Hq, lens, groups, plan, info, 152)
    return info.n_tile_wide_items > 0, info.n_row_warp_items > 0


def test_a_short_prefix_does_not_move_long_tails():
    """Long branches run as items of few rows, with a shared block or without."""
    assert layout(16, [32768] * 16, []) == (False, True)
    for blocks in (1, 2, 64):
        assert layout(16, [32768] * 16, [[0, 16, 0, blocks]]) == (True, True)
    assert layout(4, [16016] * 64, [[0, 64, 0, 1]]) == (True, True)
    assert layout(2, [4000] * 40, [[0, 40, 0, 1]]) == (True, True)


def test_small_steps_of_both_kinds_run_in_one_kernel():
    """A second kernel is not started for little work."""
    assert layout(16, [356] * 17, [[0, 17, 0, 16]]) == (True, False)
    assert layout(4, [612] * 72, [[0, 24, 0, 32], [24, 24, 0, 32],
                                  [48, 24, 0, 32]]) == (True, False)
    assert layout(2, [56] * 40, [[0, 40, 0, 1]]) == (True, False)
    # Many short tails are not little work.
    assert layout(16, [112] * 600, [[0, 600, 0, 4]]) == (True, True)


P = 1 << 20          # a pointer that no call here follows


@pytest.mark.parametrize("with_q", [True, False])
def test_appends_of_no_tokens_do_nothing(with_q):
    """A step in which no branch has new tokens: torch's empty tensors have no
    address."""
    torch = pytest.importorskip("torch")
    bf = dict(dtype=torch.bfloat16)
    ws = torch.zeros(512, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:][:256]
    table, t64 = torch.zeros(8, 64, 2), torch.zeros(8, 32, 2)
    qkv = torch.zeros(0, 6 * 128, **bf)
    q = qkv[:, :512].unflatten(1, (4, 128)) if with_q else None
    k, v = (qkv[:, a:a + 128].unflatten(1, (1, 128)) for a in (512, 640))
    row = torch.zeros(0, 576, **bf)
    qr = torch.zeros(0, 4, 192, **bf)[..., 128:] if with_q else None
    tail = (P, P, P, 0, 2, 2, 4)      # tables, lengths, row_offsets, total, nb, ..
    B.paged_rope_append(q, k, v, table, B.KV_ROPE_HALVES, q, P, P, 4, *tail, 1, 128,
                        ws)
    B.paged_rope_append_e4m3(q, k, v, table, B.KV_ROPE_PAIRS, q, P, P, P, 4, *tail,
                             1, 128, ws)
    B.paged_latent_append(row[:, :512], row[:, 512:], qr, t64, B.KV_ROPE_PAIRS, qr,
                          P, P, 4, *tail, ws)
    # What is wrong without tokens too is still refused.
    for change in (dict(block_size=8), dict(nb=0), dict(pool=None), dict(off=None)):
        a = dict(dict(pool=P, off=P, nb=2, block_size=16), **change)
        with pytest.raises(B.KVError) as e:
            B.paged_rope_append(q, k, v, table, B.KV_ROPE_HALVES, q, a["pool"], P,
                                4, P, P, a["off"], 0, a["nb"], 2, 4, 1, 128, ws,
                                block_size=a["block_size"])
        assert e.value.code == B.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("nb,Hq", [(3, 16), (5, 16), (4, 8), (4, 17), (8, 16)])
def test_a_plan_of_another_batch_is_refused(nb, Hq):
    """A step of 4 branches and 16 heads, called as one of others."""
    lens = [200, 170, 300, 165]
    plan, info = B.paged_decode_plan(4, 16, 1, 512, 20, lens, [[0, 4, 0, 10]], 152,
                                     B.KV_PLAN_LATENT)
    assert info.n_merge_rows == 4
    with pytest.raises(B.KVError) as e:
        B.paged_latent_decode_attn(P, P, P, 1000, P, P, None, 0, nb, 20, Hq, 0.1, P,
                                   P, info, P, info.workspace_bytes)
    assert e.value.code == B.KV_ERR_INVALID_ARG
    assert "does not match" in str(e.value)


NO_MEMORY = """
import resource, numpy as np
from paged_kv_cache_attn_gb300 import binding as B
n = 40_000_000
lens = np.full(n, 5, np.int32)
groups = np.zeros((0, 4), np.int32)
used = int(open("/proc/self/statm").read().split()[0]) * 4096
resource.setrlimit(resource.RLIMIT_AS, (used + (64 << 20), used + (64 << 20)))
try:
    B.paged_decode_plan(n, 1, 1, {d}, 1, lens, groups, 152, {flags})
except B.KVError as e:
    print("refused", e.code)
"""


@pytest.mark.parametrize("d,flags", [(512, B.KV_PLAN_LATENT), (128, 0)])
def test_decode_plan_without_host_memory(d, flags):
    """A plan that finds no memory is an error, not the end of the process."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(B.__file__)))
    r = subprocess.run([sys.executable, "-c", NO_MEMORY.format(d=d, flags=flags)],
                       cwd=root, capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["refused", str(B.KV_ERR_OOM)], r.stderr[-2000:]
