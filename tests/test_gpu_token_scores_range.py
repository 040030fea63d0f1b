"""The scores of rows whose largest logit over the temperature is anything that the settings allow, against the 64-bit form.
Tolerances: those of test_gpu_token_scores (their derivation holds for every distance from the maximum)."""
import pytest
import torch

from tests.test_gpu_token_scores import check, gen

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from draft_head_gb300.target import TokenScorer

BF, F32 = torch.bfloat16, torch.float32


def steps(value, down, up, V):
    """fp32 neighbours of `value`, from `down` below it to `up` above it in turn, in random order."""
    bits = torch.tensor([value], dtype=F32, device="cuda").view(torch.int32)
    at = torch.arange(V, device="cuda") % (down + up + 1) - (down if value > 0 else up)
    x = (bits + at.int()).view(F32)
    return x[torch.randperm(V, generator=gen(V + down), device="cuda")]


def score(x, tokens, T, n):
    s = TokenScorer(x.shape[0], x.shape[1], x.dtype, n)
    got = s.score(x, tokens, T)
    assert s.last_status() == 0
    check(x, tokens, T, n, got)
    return got


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1e-30, 1e-12, 1e-10, 1e-9, 1e-7, 1e-6, 1e-5, 1e-3, 100.0, 1e30, 3e38])
def test_temperatures(dt, T):
    V, rows = 9001, 8
    x = (3 * torch.randn(rows, V, generator=gen(7), device="cuda")).to(dt)
    x[1] = x[1].abs() + 7.3125
    x[2] -= 200
    x[3, ::11] = 11.6875  # ties at the maximum
    x[4] = -x[4].abs()
    x[5, 5] = 7.3125
    x[6] = 0
    T = torch.full((rows,), T, device="cuda")
    tokens = x.float().argmax(1).int()
    score(x, tokens, T, 5)
    score(x, x.float().topk(2).indices[:, 1].int(), T, 5)
    score(x, torch.randint(0, V, (rows,), generator=gen(8), device="cuda", dtype=torch.int32), T, 0)


def test_the_least_temperature():
    """1e-30 is the first that is taken."""
    x = torch.randn(2, 3000, generator=gen(9), device="cuda")
    first = torch.tensor([1e-30], device="cuda")
    T = torch.cat([first, torch.nextafter(first, torch.zeros_like(first))])
    tokens = x.argmax(1).int()
    s = TokenScorer(2, 3000, F32, 2)
    got = s.score(x, tokens, T)
    assert s.last_status() == 6
    check(x[:1], tokens[:1], T[:1], 2, type(got)(*(t[:1] for t in got)))
    for t in (got.logprob, got.entropy, got.lse, got.top_logprob):
        assert bool(torch.isnan(t[1]).all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("top", [1e10, -1e10, 1e18, 1e30, -1e30, 1e38])
def test_large_logits(dt, top):
    V = 5003
    x = torch.randn(4, V, generator=gen(10), device="cuda")
    x[0, 17] = x[0, 18] = top
    x[1] = top
    x[2] = top * (1 + torch.arange(V, device="cuda") % 3) / 4
    x[3] = top * torch.rand(V, generator=gen(11), device="cuda")
    x = x.to(dt)
    tokens = torch.tensor([18, 4000, 5, 9], dtype=torch.int32, device="cuda")
    for T in (0.5, 1.0, 2.0, 1e6, 1e8):
        score(x, tokens, torch.full((4,), T, device="cuda"), 3)
    score(x, tokens, None, 3)


# Neighbours that are about a unit apart over the temperature, where their product with log2(e) / T passes 2^24 (16,777,216).
@pytest.mark.parametrize("value,T", [(8.0, 6.88e-7), (8.0, 6.0e-7), (8.0, 8.0e-7), (8.0, 2e-7), (-8.0, 6.88e-7), (-8.0, 2e-7), (1e10, 860.0), (1e10, 200.0),
                                     (-1e10, 860.0), (1e30, 8.6e22), (2.0, 1.7e-7)])
@pytest.mark.parametrize("V", [50, 20011])
def test_neighbours_of_large_quotients(value, T, V):
    x = torch.stack([steps(value, 30, 0, V), steps(value, 3, 20, V), steps(value, 40, 40, V).sort().values, steps(value, 40, 40, V).sort(descending=True).values])
    tokens = torch.tensor([0, 7, V - 1, 20], dtype=torch.int32, device="cuda")
    score(x, tokens, torch.full((4,), T, device="cuda"), 8)


def test_results_keep_their_signs():
    """No log-probability above 0 and no entropy below it, where one token has all and its product with log2(e) / T is rounded down."""
    V = 3001
    x = torch.randn(400, V, generator=gen(12), device="cuda")
    x[torch.arange(400), torch.arange(400)] = 7.0 + torch.arange(400, device="cuda") / 64
    x[7, 100:] = 0.5
    tokens = torch.arange(400, dtype=torch.int32, device="cuda")
    for T in (1e-6, 3e-6, 1e-4, 0.01, 1.0):
        got = score(x, tokens, torch.full((400,), T, device="cuda"), 1)
        assert bool((got.logprob <= 0).all()) and bool((got.top_logprob <= 0).all()) and bool((got.entropy >= 0).all())


@pytest.mark.parametrize("T", [2.0, 4.0, 1e3, 1e37, 3e38])
def test_distances_beyond_fp32(T):
    """A logit's distance from the maximum is no fp32 number, over the temperature it is one."""
    big = torch.finfo(F32).max
    x = torch.randn(3, 4001, generator=gen(13), device="cuda")
    x[0, 5], x[0, 9] = big, -big
    x[1] = torch.linspace(-big / 2, big / 2, 4001, device="cuda") * 2
    x[2] = -big
    x[2, 4000] = big
    tokens = torch.tensor([9, 0, 17], dtype=torch.int32, device="cuda")
    got = score(x, tokens, torch.full((3,), T, device="cuda"), 32)
    if T > 2:
        assert bool(torch.isfinite(got.logprob).all())
