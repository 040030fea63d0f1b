"""Log-probabilities and ranks of given tokens, entropy and most likely tokens against their 64-bit plain form.

Tolerances, from the arithmetic (u = 2^-24): a logit's distance from the maximum, over T, is off by 3 u of itself, its
exponential by that much and 2 u (the instruction's bound), a sum of V terms by at most V / 256 + 16 additions' u; what weighs in the sum is within
2^6 of the maximum. So log-sum and log-probability are off by e = (V / 256 + 300) u and 4 u of themselves. In the entropy a
weight's error of 3 u d counts d times: sum p d^2 is at most about (log V + 4)^2. Ids and ranks are equal."""
import math

import pytest
import torch

from tests import paged_oracle as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

if torch.cuda.is_available():
    from draft_head_gb300 import binding as B
    from draft_head_gb300.target import TokenScorer

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def fp32_range(x):
    """What fp32 rounds to an infinity: from 2^128 - 2^103 on, half a step beyond its largest number. (-3.4e38 over a
    temperature of 0.5 is -6.8e38.)"""
    return math.copysign(INF, x) if abs(x) >= 2.0 ** 128 - 2.0 ** 103 else x


def check(logits, tokens, T, top_n, s):
    rows, V = logits.shape
    e = (V / 256 + 300) * U
    for r in range(rows):
        t = 1.0 if T is None else float(T[r])
        lp, rank, entropy, lse, ids, lps = P.scores(logits[r], -1 if tokens is None else int(tokens[r]), t, top_n)
        lp, lse, lps = fp32_range(lp), fp32_range(lse), torch.where(lps.abs() >= 2.0 ** 128 - 2.0 ** 103, torch.full_like(lps, -INF), lps)
        near = lambda got, want, more=0.0: got == want or abs(got - want) <= e + more + 4 * U * abs(want)  # noqa: E731
        assert near(float(s.logprob[r]), lp), (r, float(s.logprob[r]), lp)
        assert near(float(s.lse[r]), lse), (r, float(s.lse[r]), lse)
        assert near(float(s.entropy[r]), entropy, 3 * U * (math.log(V) + 4) ** 2), (r, float(s.entropy[r]), entropy)
        assert int(s.rank[r]) == rank, (r, int(s.rank[r]), rank)
        assert torch.equal(s.top_ids[r], ids), (r, s.top_ids[r].tolist(), ids.tolist())
        got = s.top_logprob[r].double()
        assert bool(((got == lps) | ((got - lps).abs() <= e + 4 * U * lps.abs())).all()), (r, got, lps)


CASES = [
    # dtype, rows, V, top_n
    (F32, 1, 1, 1), (F32, 3, 2, 2), (BF, 2, 7, 3), (F32, 5, 33, 32), (BF, 4, 31, 32), (F32, 2, 1000, 20), (BF, 7, 4097, 5),
    (F32, 3, 8193, 1), (BF, 40, 32000, 8), (F32, 1, 151936, 20), (BF, 1, 151936, 32), (BF, 9, 50257, 20), (F32, 6, 50257, 0),
    (F32, 300, 3001, 4), (BF, 1300, 2050, 8), (F32, 700, 20000, 2), (BF, 1, 2000003, 8),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_scores(case):
    dt, rows, V, n = CASES[case]
    g = gen(case)
    x = 2.0 * torch.randn(rows, V, generator=g, device="cuda")
    if V > 100:
        x.scatter_add_(1, torch.randint(0, V, (rows, 30), generator=g, device="cuda"), 12 * torch.rand(rows, 30, generator=g, device="cuda"))
    x = x.to(dt)
    tokens = torch.randint(-1, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tokens[::3] = x[::3].argmax(1).int()
    T = 0.25 + 2 * torch.rand(rows, generator=g, device="cuda")
    s = TokenScorer(rows, V, dt, n)
    got = s.score(x, tokens, T)
    assert s.last_status() == 0
    pick = list(range(rows)) if rows <= 40 else list(range(0, rows, max(1, rows // 40)))
    check(x[pick], tokens[pick], T[pick], n, type(got)(*(t[pick] for t in got)))
    again = TokenScorer(rows, V, dt, n).score(x, tokens, T)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # Without tokens and temperatures: none, and 1.
    got = s.score(x)
    check(x[pick], None, None, n, type(got)(*(t[pick] for t in got)))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [1, 5, 32])
def test_special_rows(dt, n):
    V = 9000
    low = float(torch.finfo(dt).min)
    base = torch.randn(V, generator=gen(n), device="cuda")
    rows, tokens = [], []

    def row(x, *toks):
        for t in toks:
            rows.append(x.clone())
            tokens.append(t)

    row(torch.zeros(V, device="cuda"), 0, 1, 4500, V - 1, -1)              # all alike
    row(torch.full((V,), -INF, device="cuda"), 0, 17, V - 1)               # nothing above -inf
    row(torch.full((V,), low, device="cuda"), 0, 8000)                     # the type's lowest everywhere
    few = torch.full((V,), -INF, device="cuda")
    few[[3, 4444, 8999]] = torch.tensor([1.0, -2.0, 1.0], device="cuda")
    row(few, 3, 4444, 8999, 5000, 0, V - 2)                                # a mask that leaves three
    few = torch.full((V,), low, device="cuda")
    few[[7, 6001]] = torch.tensor([5.0, -INF], device="cuda")
    row(few, 7, 6001, 6002, 6, 8)                                          # lowest values above an infinity
    x = base.clone()
    x[[10, 5000, 8998]] = INF
    row(x, 10, 5000, 8998, 11, 0)                                          # infinities share everything
    x = base.clone()
    x[::7] = NAN
    x[1::7] = -INF
    row(x, 0, 1, 2, 8995, 8996)                                            # NaN counts as -inf
    x = base.clone()
    x[1234] = float(torch.finfo(dt).max)
    row(x, 1234, 0)                                                        # the type's largest
    row(torch.arange(V, device="cuda").float() / 64, V - 1, 0, 4000)       # rising: every token is the best so far
    row(-torch.arange(V, device="cuda").float() / 64, V - 1, 0, 4000)
    row((torch.arange(V, device="cuda") % 3 == 0).float(), 0, 1, 2, 8997, 8999)  # ties
    x = base.clone()
    x[77] = 60.0
    row(x, 77, 78)                                                         # one token has nearly all: entropy near 0
    row(-base.abs() * 0.0, 5)                                              # negative zeros among zeros tie with them
    x = torch.stack(rows).to(dt)
    tokens = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    for T in (None, torch.full((len(rows),), 0.5, device="cuda")):
        s = TokenScorer(len(rows), V, dt, n)
        got = s.score(x, tokens, T)
        assert s.last_status() == 0
        check(x, tokens, T, n, got)


@pytest.mark.parametrize("V", [1, 2, 3])
def test_rows_of_a_few_tokens(V):
    """More places than tokens: the rest are -1 and -inf."""
    x = torch.randn(4, V, generator=gen(V), device="cuda")
    s = TokenScorer(4, V, F32, 6)
    got = s.score(x, torch.zeros(4, dtype=torch.int32, device="cuda"))
    check(x, [0] * 4, None, 6, got)
    assert bool((got.top_ids[:, V:] == -1).all()) and bool((got.top_logprob[:, V:] == -INF).all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [50257, 131])
def test_rows_at_any_alignment(dt, V):
    """Rows apart by more than V, from any element on, beside NaN."""
    g = gen(V)
    x = (3 * torch.randn(9, V, generator=g, device="cuda")).to(dt)
    tokens = torch.randint(0, V, (9,), generator=g, device="cuda", dtype=torch.int32)
    want = None
    for skew in (0, 1, 3, 6):
        wide = torch.full((9, V + 13), NAN, dtype=dt, device="cuda")
        wide[:, skew:skew + V] = x
        view = wide[:, skew:skew + V]
        got = TokenScorer(9, V, dt, 4).score(view, tokens)
        check(x, tokens, None, 4, got)
        if want is not None:
            assert torch.equal(want.rank, got.rank) and torch.equal(want.top_ids, got.top_ids)
        want = got


def test_settings_that_are_reported():
    x = torch.randn(6, 500, generator=gen(1), device="cuda")
    T = torch.tensor([1.0, 0.0, -1.0, NAN, INF, 0.7], device="cuda")
    tokens = torch.tensor([3, 3, 3, 3, 3, 3], dtype=torch.int32, device="cuda")
    s = TokenScorer(6, 500, F32, 3)
    got = s.score(x, tokens, T)
    assert s.last_status() == 6 and s.last_status() == 0
    for t in (got.logprob, got.entropy, got.lse):
        assert bool(torch.isnan(t[1:5]).all()) and not bool(torch.isnan(t[[0, 5]]).any())
    assert bool(torch.isnan(got.top_logprob[1:5]).all())
    check(x[[0, 5]], tokens[[0, 5]], T[[0, 5]], 3, type(got)(*(t[[0, 5]] for t in got)))
    tokens = torch.tensor([500, -2, 2 ** 31 - 1, -2 ** 31, 499, 0], dtype=torch.int32, device="cuda")
    got = s.score(x, tokens)
    assert s.last_status() == 6 and s.last_status() == 0
    assert bool(torch.isnan(got.logprob[:4]).all()) and bool((got.rank[:4] == -1).all())
    assert not bool(torch.isnan(got.entropy).any())
    check(x[4:], tokens[4:], None, 3, type(got)(*(t[4:] for t in got)))
    # With T outside its range and a token given too.
    got = s.score(x, torch.full((6,), -1, dtype=torch.int32, device="cuda"), T)
    assert s.last_status() == 6
    assert bool(torch.isnan(got.logprob[1:5]).all()) and float(got.logprob[0]) == 0.0


def test_results_that_nobody_wants():
    """Every output may be left out."""
    x = torch.randn(3, 700, generator=gen(2), device="cuda")
    tokens = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    want = TokenScorer(3, 700, F32, 4).score(x, tokens)
    ws = B.workspace(256)
    for left_out in range(6):
        out = [torch.empty_like(t) for t in want]
        B.domino_token_logprobs(x, 3, 700, tokens, None, 4, *(None if i == left_out else t for i, t in enumerate(out)), ws)
        assert all(i == left_out or torch.equal(a, b) for i, (a, b) in enumerate(zip(out, want)))
    B.domino_token_logprobs(x, 3, 700, tokens, None, 0, None, None, None, None, None, None, ws)
    assert B.domino_last_status(ws) == 0


@pytest.mark.parametrize("rows,V", [(1, 151936), (64, 4000)])
def test_on_another_stream_and_in_a_graph(rows, V):
    g = gen(rows)
    x = torch.randn(rows, V, generator=g, device="cuda").to(BF)
    other = torch.randn(rows, V, generator=g, device="cuda").to(BF)
    tokens = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    want = [type(s)(*(t.clone() for t in s)) for s in (TokenScorer(rows, V, BF, 8).score(y, tokens) for y in (x, other))]
    s = TokenScorer(rows, V, BF, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.score(x, tokens)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.score(x, tokens)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    x.copy_(other)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


@pytest.mark.slow
def test_offsets_pass_32_bits():
    """Rows that begin past element 2^31."""
    rows, V = 3, 40000
    stride = 2 ** 30 + 8
    pool = torch.empty(2 * stride + V, dtype=BF, device="cuda")
    x = pool.as_strided((rows, V), (stride, 1))
    x.copy_(torch.randn(rows, V, generator=gen(3), device="cuda"))
    tokens = torch.tensor([1, 39999, 20000], dtype=torch.int32, device="cuda")
    check(x, tokens, None, 8, TokenScorer(rows, V, BF, 8).score(x, tokens))
