"""Beam selection against its definition in 64 bits, and with the pool's branches."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_attn_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


def call(x, scores, groups, beams, n, ws_fill=0xA5):
    ws = torch.full((B.kv_beam_select_workspace_size(groups, beams, x.shape[1], n),),
                    ws_fill, dtype=torch.uint8, device="cuda")
    out = (torch.full((groups, n), 55.0, device="cuda"),
           torch.full((groups, n), 55, dtype=torch.int32, device="cuda"),
           torch.full((groups, n), 55, dtype=torch.int32, device="cuda"))
    B.kv_beam_select(x, scores, groups, beams, n, *out, ws)
    return out


def want(x, scores, groups, beams, n):
    """(scores in 64 bits, parents, tokens), ties to the lower (beam, token)."""
    V = x.shape[1]
    x = x.double()
    x = torch.where(x.isnan(), -math.inf, x)
    lse = torch.logsumexp(x, 1, keepdim=True)
    y = scores.double()[:, None] + (x - lse)
    ok = (scores > -math.inf)[:, None] & (x > -math.inf) & lse.isfinite()
    y = torch.where(ok, y, -math.inf).view(groups, beams * V)
    best, at = torch.sort(y, dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    if best.shape[1] < n:
        pad = n - best.shape[1]
        best = torch.nn.functional.pad(best, (0, pad), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, pad))
    none = best == -math.inf
    return best, torch.where(none, -1, at // V).int(), \
        torch.where(none, -1, at % V).int()


def check(x, scores, groups, beams, n):
    got, ref = call(x, scores, groups, beams, n), want(x, scores, groups, beams, n)
    # A result is the score plus the logit less the log of the sum, in 64 bits from
    # sums of at most 32 exponentials in fp32: each of those 2^-21 (its argument's
    # rounding, up to 2^-23 x 1.45 (x - max) where it counts, and 2^-22 of the
    # function), 32 additions of 2^-24 each: 2^-18 of the sum at the very most, as
    # much of the logarithm; then rounded to fp32 (2^-24).
    ref_s = ref[0].nan_to_num(neginf=0.0)
    err = (got[0].double().nan_to_num(neginf=0.0) - ref_s).abs()
    assert torch.equal(got[0] == -math.inf, ref[0] == -math.inf)
    assert (err <= 2.0 ** -18 + ref_s.abs() * 2.0 ** -24).all()
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])


def make(groups, beams, V, dtype, seed=1, gain=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(groups * beams, V, generator=g, device="cuda") * gain).to(dtype)
    s = torch.randn(groups * beams, generator=g, device="cuda") * 2 - 30
    return x, s


DT = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("groups,beams,V,n", [
    (1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 5, 15), (1, 4, 2047, 8), (1, 4, 2048, 8),
    (3, 4, 2049, 8), (1, 8, 32000, 16), (5, 3, 50257, 6), (40, 8, 12345, 16),
    (1, 1, 151936, 128), (300, 4, 8192, 4), (300, 4, 8193, 128), (2, 64, 1000, 128),
    (1, 1000, 130, 50)])
def test_sizes(groups, beams, V, n, dtype):
    check(*make(groups, beams, V, dtype), groups, beams, n)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_rows_apart_and_unaligned(pad, dtype):
    x, s = make(2, 4, 5003 + pad, dtype, 2)
    for start in range(pad):
        view = x[:, start:start + 5003]
        check(view, s, 2, 4, 9)


@pytest.mark.parametrize("dtype", DT)
def test_ties(dtype):
    """Equal logits in a beam, equal beams, and logits that are all the same (more
    candidates than fit)."""
    x, s = make(2, 4, 9000, dtype, 3)
    x = (x * 2).round() / 2
    check(x, s, 2, 4, 40)
    x[1::2] = x[0::2]
    s[1::2] = s[0::2]
    check(x, s, 2, 4, 40)
    x[:] = 1.5
    check(x, s, 2, 4, 40)
    x = torch.zeros(300 * 4, 8200, dtype=dtype, device="cuda")
    s = torch.zeros(300 * 4, device="cuda")
    check(x, s, 300, 4, 100)


@pytest.mark.parametrize("dtype", DT)
def test_beams_and_tokens_that_are_not_there(dtype):
    """First steps (one beam), finished beams, masked tokens, too few of them."""
    x, s = make(4, 5, 3001, dtype, 4)
    s[1:5] = -math.inf                 # one beam alone
    s[5:10] = -math.inf                # a group without any
    s[12] = float("nan")
    x[15:20, 4:] = -math.inf           # four tokens a beam
    x[16] = -math.inf                  # a beam that cannot go on
    x[18, 2] = float("nan")
    x[13, 100:3000] = float("-inf")
    check(x, s, 4, 5, 25)
    check(x, s, 4, 5, 1)
    x[10, 7] = math.inf
    check(x, s, 4, 5, 25)


@pytest.mark.parametrize("dtype", DT)
def test_logits_of_all_sizes(dtype):
    for gain, shift in ((1e-6, 0.0), (40.0, 0.0), (1.0, 1000.0), (1.0, -1000.0),
                        (1e30, 0.0)):
        x, s = make(2, 3, 7001, dtype, 5)
        x = (x.double() * gain + shift).to(dtype)
        ref = want(x, s, 2, 3, 6)
        got = call(x, s, 2, 3, 6)
        assert torch.equal(got[2], ref[2]) and torch.equal(got[1], ref[1])


def test_sorted_and_reversed_logits():
    """The highest logits all in the first piece, or the last."""
    x = torch.linspace(-8, 8, 40000, device="cuda").repeat(3, 1)
    s = torch.tensor([-1.0, -1.1, -1.7], device="cuda")
    check(x, s, 1, 3, 64)
    check(x.flip(1).contiguous(), s, 1, 3, 64)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [5, 128])
def test_rows_whose_candidates_lie_together(dtype, n):
    """Equal logits all over a long row, and masked rows with one run of tokens that
    may follow: more candidates than fit, of few threads or of all."""
    V = 151936
    x = torch.full((3, V), -math.inf, dtype=dtype, device="cuda")
    x[0] = 0.25
    g = torch.Generator(device="cuda").manual_seed(7)
    x[1, 70001:73001] = torch.randn(3000, generator=g, device="cuda").to(dtype)
    x[2, 151000:] = -2.0
    x[2, 5] = -1.0
    s = torch.tensor([-1.0, -3.0, -2.0], device="cuda")
    check(x, s, 1, 3, n)
    check(x, s, 3, 1, n)
    check(x[1:, 70000:], s[1:], 2, 1, n)


@pytest.mark.parametrize("dtype", DT)
def test_equal_results_of_many_beams(dtype):
    """More equal results than fit, over the beams of a group."""
    x = torch.zeros(64, 40000, dtype=dtype, device="cuda")
    x[:, 20000:] = -3.0
    s = torch.zeros(64, device="cuda")
    check(x, s, 2, 32, 128)
    x[:, ::2] = 1.0
    check(x, s, 2, 32, 60)
    s[3::7] = 0.5
    check(x, s, 2, 32, 60)
    check(x[:1], s[:1], 1, 1, 128)


@pytest.mark.parametrize("dtype", DT)
def test_logits_that_rise_along_the_row(dtype):
    """References that move in some threads, by more than exponentials can hold."""
    x = torch.randn(640, 20000, device="cuda") * 2
    x += torch.arange(20000, device="cuda") // 1500 * 45.0
    x[1::2, :9000] = -math.inf
    x[2::4, 11000:] -= 900.0
    s = torch.linspace(-3, -1, 640, device="cuda")
    check(x.to(dtype), s, 160, 4, 12)


def test_captured_and_same_every_time():
    x, s = make(6, 8, 32003, torch.bfloat16, 6)
    ws = torch.zeros(B.kv_beam_select_workspace_size(6, 8, 32003, 16),
                     dtype=torch.uint8, device="cuda")
    out = (torch.zeros(6, 16, device="cuda"),
           torch.zeros(6, 16, dtype=torch.int32, device="cuda"),
           torch.zeros(6, 16, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.kv_beam_select(x, s, 6, 8, 16, *out, ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.kv_beam_select(x, s, 6, 8, 16, *out, ws)
    x.copy_(make(6, 8, 32003, torch.bfloat16, 7)[0])
    first = call(x, s, 6, 8, 16)
    for _ in range(4):
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, f in zip(out, first):
            assert torch.equal(o, f)
    check(x, s, 6, 8, 16)


def test_behind_a_join_of_streams():
    """Logits that another stream makes, late, eager and captured: the first launch
    starts early, but reads nothing before."""
    x, s = make(4, 4, 30000, torch.float32, 9)
    slow = torch.randn(4096, 4096, device="cuda")
    logits, scores = torch.empty_like(x), torch.empty_like(s)
    ws = torch.empty(B.kv_beam_select_workspace_size(4, 4, 30000, 8), dtype=torch.uint8,
                     device="cuda")
    out = (torch.empty(4, 8, device="cuda"),
           torch.empty(4, 8, dtype=torch.int32, device="cuda"),
           torch.empty(4, 8, dtype=torch.int32, device="cuda"))
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.mm(slow, slow)
            logits.copy_(x)
        scores.copy_(s)
        here.wait_stream(side)
        B.kv_beam_select(logits, scores, 4, 4, 8, *out, ws)
        logits.fill_(0.0)
        scores.fill_(-1.0)

    def good():
        torch.cuda.synchronize()
        ref = want(x, s, 4, 4, 8)
        assert torch.equal(out[1], ref[1]) and torch.equal(out[2], ref[2])
        for o in out:
            o.zero_()

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        step()
        good()
        step()
    good()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for _ in range(3):
        graph.replay()
        graph.replay()
        good()


def test_a_search_on_the_pool():
    """Steps of a beam search: selection, the branches reordered with their caches,
    the new tokens appended, each beam's cache that of its own tokens."""
    Hkv, d, nblk, V, beams = 2, 64, 200, 500, 4
    k = torch.zeros(1, nblk, Hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    pool = B.kv_pool_create(nblk, 1, Hkv, d, k, v)
    emb = torch.randn(V, Hkv, d, device="cuda").bfloat16()
    root = B.kv_branch_create(pool)
    prompt = list(range(37))
    B.kv_append(pool, root, 37, emb[prompt][None].contiguous(),
                -emb[prompt][None].contiguous())
    ids = [root] + [-1] * (beams - 1)
    seqs = [prompt] + [None] * (beams - 1)
    scores = torch.full((beams,), -math.inf, device="cuda")
    scores[0] = 0.0
    g = torch.Generator(device="cuda").manual_seed(8)
    for step in range(20):
        x = torch.randn(beams, V, generator=g, device="cuda") * 2
        ref = want(x, scores, 1, beams, beams)
        scores, parents, tokens = (o[0] for o in call(x, scores, 1, beams, beams))
        assert torch.equal(parents, ref[1][0]) and torch.equal(tokens, ref[2][0])
        live = [i for i in ids if i >= 0]
        at = {b: j for j, b in enumerate(live)}
        place = [at[ids[p]] for p in parents.tolist()]
        ids = B.kv_beam_reorder(pool, live, place)
        assert len(set(ids)) == beams
        seqs = [seqs[p] + [t] for p, t in zip(parents.tolist(), tokens.tolist())]
        new = emb[tokens.long()][None].contiguous()
        B.kv_append_batch(pool, ids, [1] * beams, new, -new)
        torch.cuda.synchronize()
        for b, seq in zip(ids, seqs):
            table, L = B.kv_get_block_table(pool, b)
            assert L == len(seq)
            t = torch.as_tensor(np.asarray(table), dtype=torch.long, device="cuda")
            rows = k[0][t].transpose(1, 2).reshape(-1, Hkv, d)[:L]
            assert torch.equal(rows, emb[seq])
            assert torch.equal(v[0][t].transpose(1, 2).reshape(-1, Hkv, d)[:L],
                               -emb[seq])
    B.kv_pool_destroy(pool)
