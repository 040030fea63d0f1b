"""Attention where scores are so large that only the slots that tie for a row's maximum count (products of queries and keys beyond
2^24): over the cache in one piece and in pages, by few rows and by many.

The scores are exact in fp32 (powers of two times small integers), so the output is the mean of the tying slots' values, to within the
output's rounding and that of their weights (2^-8 and 2^-8 of bf16's values), and the log-sum that of their number above the maximum,
to within 4 units of fp32."""
import math

import pytest
import torch

from tests import paged_oracle as P
from tests.test_gpu_paged import BF, E4M3, F32, H, U, gen, ints, layer, randn

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from draft_head_gb300.target import BlockAttention

HQ, HKV, CTX = 4, 2, 400


def expect(q0, k0, v, scale, seen):
    """q0, k0: the one element that queries and keys have; v [slots, D]; seen: the number of slots."""
    s = (k0[:seen].double() * float(q0)) * scale
    top = s == s.max()
    return v[:seen][top].double().mean(0), float(s.max()) + math.log(int(top.sum()))


@pytest.mark.parametrize("kind", [E4M3, BF, F32, "whole"])
@pytest.mark.parametrize("n", [1, 4, 16, 200])
@pytest.mark.parametrize("power", [10, 28, 31, 33, 100])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 128])
def test_only_ties_count(kind, n, power, sign, D):
    ties(kind, n, power, sign, D, 0.125)


@pytest.mark.parametrize("kind", [E4M3, BF, F32, "whole"])
@pytest.mark.parametrize("n", [1, 4, 16, 200])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", [0.9, 1.0])
def test_scores_next_to_the_end_of_the_range(kind, n, sign, scale):
    """Up to 2^127.7 in powers of two."""
    ties(kind, n, 124, sign, 64, scale)


def ties(kind, n, power, sign, D, scale):
    g = gen(n + power)
    pages = P.Pages(BF if kind == "whole" else kind, [CTX + n], HKV, 32, D, n + power)
    # Keys 1 to 3 at element 0 (all of one sign, so that the maximum is the largest or the smallest product), 0 elsewhere.
    k0 = torch.randint(1, 4, (CTX + n,), generator=g, device="cuda").float()
    for s in range(CTX + n):
        k = torch.zeros(1, D, device="cuda")
        k[0, 0] = float(k0[s])
        pages.put("k", 0, s, k)
    q0 = sign * 3.0 * 2.0 ** power  # steps between scores: 3 * 2^power / 8 and more
    q = torch.zeros(n, HQ, D, device="cuda")
    q[:, :, 0] = q0
    q = q.to(pages.rows_type)
    p = layer(pages, HQ, n, n, CTX, scale=scale)
    if kind == "whole":
        k, v = (torch.zeros(1, HKV, 640, D, dtype=BF, device="cuda") for _ in "kv")
        p.read(k, v, ints([CTX + n]))
        p = BlockAttention(k, v, HQ, n, n, CTX, scale=scale)
    out, lse = p.attend(q, ints([CTX]), want_lse=True)
    assert p.last_status() == 0
    h = H if kind != F32 else 0.0
    for h_kv in range(HKV):
        v = pages.values("v", 0, CTX + n)[h_kv]
        for i in range(0, n, max(1, n // 10)):
            want, wl = expect(q0, k0, v, scale, CTX + i + 1)
            tol = 2 * h * v.abs().max() + (CTX + n) * U * v.abs().max()
            for head in range(h_kv * HQ // HKV, (h_kv + 1) * HQ // HKV):
                assert bool(((out[i, head].double() - want).abs() <= tol).all()), (i, head)
                assert abs(float(lse[i, head]) - wl) <= 4 * U * abs(wl) + 1e-4, (float(lse[i, head]), wl)


@pytest.mark.parametrize("kind", [E4M3, BF, F32])
@pytest.mark.parametrize("n", [1, 4, 16, 200])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 16, 2.0 ** 24, 2.0 ** 50])
def test_large_scores_of_any_kind(kind, n, size):
    """Outputs lie among the values, and the log-sum at the largest score, to within what fp32 gives of a score."""
    pages = P.Pages(kind, [CTX + n], HKV, 32, 64, n)
    q = (size * randn(gen(n), n, HQ, 64)).to(pages.rows_type)
    if kind != E4M3:
        pages.k.mul_(2.0 ** 14)
    else:
        pages.k_scale.add_(14)
    p = layer(pages, HQ, n, n, CTX)
    out, lse = p.attend(q, ints([CTX]), want_lse=True)
    assert p.last_status() == 0
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for i in range(0, n, max(1, n // 10)):
        k, v = (pages.values(x, 0, CTX + i + 1).repeat_interleave(HQ // HKV, 0) for x in "kv")
        room = 2 * H * v.abs().amax(1)
        assert bool((out[i].double() <= v.amax(1) + room).all()) and bool((out[i].double() >= v.amin(1) - room).all())
        s = torch.einsum("hsd,hd->hs", k, q[i].double()) * p.scale
        big = float(torch.einsum("hsd,hd->hs", k.abs(), q[i].double().abs()).max() * p.scale)
        assert bool(((lse[i].double() - torch.logsumexp(s, 1)).abs() <= 2 * 68 * U * big + 1e-4).all())
