"""Attention over quantised pages whose values are anything that their scales can stand for, against the 64-bit form on what codes and
scales stand for. Tolerances: those of test_gpu_paged."""
import pytest
import torch

from tests import paged_oracle as P
from tests.test_gpu_paged import E4M3, check, gen, ints, run

pytestmark = pytest.mark.gpu


def vector(seed, hkv, D, e):
    """[hkv, D] whose scale is 2^e: largest magnitude in (224, 448] 2^e, below 2^128."""
    x = torch.rand(hkv, D, generator=gen(seed), device="cuda", dtype=torch.float64) * 2 - 1
    x[:, 0] = 1.0
    return x * 240.0 * 2.0 ** e


def large(slots):
    def prepare(pages, q):
        q.mul_(0.05)  # scores close to one another: the maximum does not grow, so no product passes fp32's range
        for i, (s, e) in enumerate(slots):
            pages.put("v", 0, s, vector(i, pages.k.shape[1], pages.k.shape[3], e))
            at = pages.table[0, s // pages.page].long()
            assert bool((pages.v_scale[at, :, s % pages.page] == e + 127).all())
    return prepare


# Packed rows of a kv head: 2, 8, 16, 32, 400.
@pytest.mark.parametrize("n", [1, 4, 8, 16, 200])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [90, 97, 100, 104, 110, 115, 116, 117, 118, 119, 120])
def test_a_large_value(n, D, e):
    spec = ([n, n], [130, 77], 4, 2, D, "causal", 0, 0, False, 16)
    check(spec, *run(E4M3, spec, 50 + e, prepare=large([(40, e)])))


@pytest.mark.parametrize("n", [1, 4, 8])
@pytest.mark.parametrize("ctx", [130, 2500])
def test_large_values_everywhere_few_rows(n, ctx):
    """Up to 16 packed rows: sums of weights and of products that pass neither end of fp32's range, with as many large values as there are
    slots, and scores of any kind."""
    spec = ([n], [ctx], 4, 2, 64, "causal", 0, 0, False, 32)

    def prepare(pages, q):
        pages.v_scale.fill_(246)  # 2^119
        pages.v_scale[::3] = 240

    check(spec, *run(E4M3, spec, 77, prepare=prepare))


@pytest.mark.parametrize("n", [1, 4, 8])
@pytest.mark.parametrize("e", [100, 115, 119])
@pytest.mark.parametrize("gap", [-12, -8, 3, 6, 12, 40, 100, 140])
def test_weights_beside_large_values(n, e, gap):
    """The softmax's sum is that of all slots, where the one with the largest weight times value has little of it: its score is `gap`
    below the others' (in powers of two)."""
    D = 64
    spec = ([n], [300], 2, 1, D, "full", 0, 0, False, 16)

    def prepare(pages, q):
        q.zero_()
        q[:, :, 0] = 8.0
        for s in range(300 + n):
            k = torch.zeros(1, D, device="cuda")
            k[0, 0] = -gap / 1.4426950408889634 if s == 55 else 0.25 * (s % 3)  # scale D^-0.5 = 1/8: the score itself
            pages.put("k", 0, s, k)
        pages.put("v", 0, 55, vector(3, 1, D, e))

    check(spec, *run(E4M3, spec, 78, prepare=prepare))


@pytest.mark.parametrize("n", [1, 4, 8, 16, 200])
def test_the_smallest_values(n):
    """Scales of 2^-100, alone and beside others: what reaches bf16's normal numbers is right."""
    spec = ([n], [300], 4, 2, 64, "causal", 0, 0, False, 16)

    def prepare(pages, q):
        pages.v_scale.fill_(27)
        pages.v_scale[1::2] = 40

    q, pages, p, seen, st, out, lse = run(E4M3, spec, 79, prepare=prepare)
    check(spec, q, pages, p, seen, st, out, lse)
    want = torch.stack([torch.softmax(torch.einsum("hsd,hd->hs", pages.values("k", 0, 300 + n).repeat_interleave(2, 0)[:, :301 + i], q[i].double()) * p.scale, -1)
                        .unsqueeze(1).matmul(pages.values("v", 0, 300 + n).repeat_interleave(2, 0)[:, :301 + i])[:, 0] for i in range(n)])
    assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -7


@pytest.mark.parametrize("kind", [E4M3, torch.bfloat16, torch.float32])
def test_read_into_the_largest_capacity(kind):
    """2^31 - 1 slots (in one place, a stride of 0): as many as the layer takes."""
    from tests.test_gpu_paged import layer
    pages = P.Pages(kind, [40], 2, 16, 64, 4)
    p = layer(pages, 2, 1, 1, 30)
    out = [torch.full((1, 2, 1, 64), 7.0, dtype=pages.rows_type, device="cuda").expand(1, 2, 2 ** 31 - 1, 64) for _ in "kv"]
    p.read(*out, ints([1]), first=ints([37]))
    assert p.last_status() == 0
    for which, o in zip("kv", out):
        assert torch.equal(o[0, :, 0].double(), pages.values(which, 0, 40)[:, 37])
    p.read(*out, ints([2 ** 31 - 1]))
    assert p.last_status() == 6


@pytest.mark.parametrize("n", [1, 4, 8, 16, 200])
@pytest.mark.parametrize("query,byte", [(95, 27), (112, 27), (116, 27), (118, 27), (-110, 235), (-118, 244)])
def test_queries_and_keys_of_unlike_sizes(n, query, byte):
    """Large queries over small keys and the other way round: their product is a number."""
    spec = ([n], [300], 4, 2, 64, "causal", 0, 0, False, 16)

    def prepare(pages, q):
        pages.k_scale.fill_(byte)
        q.mul_(2.0 ** query)

    q, pages, p, seen, st, out, lse = run(E4M3, spec, 81, prepare=prepare)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check(spec, q, pages, p, seen, st, out, lse)


@pytest.mark.parametrize("n", [1, 4, 8, 16, 200])
def test_queries_below_the_normal_numbers(n):
    """Rows whose largest element is subnormal (below 2^-126), over keys next to bf16's largest."""
    spec = ([n], [300], 4, 2, 64, "causal", 0, 0, False, 16)

    def prepare(pages, q):
        pages.k_scale.fill_(246)
        q.mul_(2.0 ** -100).mul_(2.0 ** -30)
        assert 0 < float(q.abs().max()) < 2.0 ** -126

    q, pages, p, seen, st, out, lse = run(E4M3, spec, 82, prepare=prepare)
    check(spec, q, pages, p, seen, st, out, lse)
