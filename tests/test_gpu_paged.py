"""The operators on a cache in pages against their 64-bit plain forms: keys and values normed, rotated and quantised into
pages, read back, and attention of a chunk of rows over them.

Tolerances, from the arithmetic (u = 2^-24 the fp32 unit, h = 2^-8 the bf16 one):
- a code stands for its value within half a step of the grid (of the exponent, or of the smallest one), and norm and rotation
  are off by 32 u of the pair's magnitude as in the cache in one piece; values are quantised as they are, so their codes and
  scales are equal to the plain form's;
- reading back is exact;
- attention as over the cache in one piece, on what the codes stand for: they and their scales are exact in bf16.
"""
import pytest
import torch

from tests import paged_oracle as P
from tests import target_oracle as O

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8

if torch.cuda.is_available():
    from draft_head_gb300 import binding as B
    from draft_head_gb300.target import BlockAttention, PagedAttention, rope_table

BF, F32, E4M3 = torch.bfloat16, torch.float32, "e4m3"
KINDS = [E4M3, BF, F32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return s


def numbers(x):
    """Comparable by torch.equal."""
    return x.nan_to_num(1e30, 2e30, -2e30)


def layer(pages, hq, max_tokens, max_q, max_ctx, **kw):
    return PagedAttention(pages.k, pages.v, pages.table, hq, max_tokens, max_q, max_ctx, k_scale=pages.k_scale,
                          v_scale=pages.v_scale, **kw)


# ---------------------------------------------------------------------------
# Into the pages.
# ---------------------------------------------------------------------------
APPEND = [
    # kind, page, rows per request, ctx, hq, hkv, D, rot, interleaved, slot_major, norm, weights, positions
    (E4M3, 16, [16], [5], 32, 8, 128, 128, False, False, True, True, False),
    (E4M3, 64, [1], [0], 4, 1, 64, 64, False, True, True, True, False),
    (E4M3, 32, [3, 0, 40, 1], [0, 9, 30, 31], 10, 2, 80, 80, False, False, True, True, True),
    (E4M3, 16, [7, 2], [1, 40], 6, 3, 96, 40, True, True, False, False, False),
    (E4M3, 128, [5, 5], [0, 3], 4, 4, 256, 128, False, False, True, False, True),
    (E4M3, 16, [9, 4], [3, 3], 8, 2, 16, 0, False, False, False, False, False),
    (E4M3, 256, [5], [250], 0, 2, 48, 48, True, False, True, True, False),
    (E4M3, 16, [2000, 1, 1300, 0, 900], [0, 100, 7, 3, 15], 32, 8, 128, 128, False, False, True, True, False),
    (E4M3, 64, [1500, 1500], [0, 33], 5, 1, 64, 32, True, True, False, False, True),
    (E4M3, 32, [700] * 4, [1, 2, 3, 4], 14, 2, 80, 20, False, False, True, True, False),
    (BF, 16, [16, 3], [5, 14], 8, 2, 128, 128, False, True, True, True, False),
    (BF, 32, [5, 5], [0, 30], 8, 2, 72, 0, False, False, False, False, False),
    (BF, 64, [1900, 800], [0, 60], 32, 8, 128, 64, True, False, False, False, False),
    (F32, 16, [7, 2], [1, 40], 6, 3, 80, 40, True, True, True, True, False),
    (F32, 128, [1700, 1600], [0, 3], 4, 4, 256, 12, False, False, True, False, True),
]


def plain_turned(x, weight, eps, table, pos, rot, pairs, norm):
    if norm:
        return O.norm_rope(x, weight, eps, table, pos, rot, pairs)
    x = x.to(O.F64)
    out = x.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
        c, s = table[pos.long(), j].to(O.F64)[:, None], table[pos.long(), rot // 2 + j].to(O.F64)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def check_codes(codes, scale, want, err):
    """codes [n, hkv, D] and scales [n, hkv] hold `want` (float64, known to `err`) by the definition."""
    got = P.dequantise(codes, scale)
    e = scale.to(torch.int32) - 127
    unit = P.pow2(e)
    most = want.abs().amax(-1)
    assert bool((most <= 448 * unit + err).all())
    assert bool(((most > 224 * unit - err) | (e == -100)).all())
    y = (want.abs() / unit[..., None]).clamp(min=2.0 ** -6)
    step = P.pow2(torch.floor(torch.log2(y)).int() - 3) * unit[..., None]
    assert bool(((got - want).abs() <= step / 2 * 1.0001 + err).all())


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case):
    kind, page, rows, ctx, hq, hkv, D, rot, pairs, slot_major, norm, weights, given = APPEND[case]
    g = gen(100 + case)
    b, st = len(rows), starts(rows)
    pages = P.Pages(kind, [r + c for r, c in zip(rows, ctx)], hkv, page, D, case, slot_major)
    dt = pages.rows_type
    before = [pages.k.clone(), pages.v.clone()] + [s.clone() for s in (pages.k_scale, pages.v_scale) if s is not None]
    top = max(r + c for r, c in zip(rows, ctx)) + 50
    qkv = (1.7 * randn(g, st[-1], (hq + 2 * hkv) * D)).to(dt)
    table = rope_table(top, rot) if rot else None
    qw, kw = ((1 + 0.3 * randn(g, D)).to(dt), (1 + 0.3 * randn(g, D)).to(dt)) if weights else (None, None)
    pos = [c + i for n, c in zip(rows, ctx) for i in range(n)]
    if given:
        pos = [(p * 7 + 3) % top for p in pos]
    p = layer(pages, hq or hkv, st[-1], max(rows), max(ctx), rope=table, norm=norm, q_weight=qw, k_weight=kw, eps=1e-5,
              interleaved=pairs)
    if hq:
        q = p.append(qkv, ints(ctx), q_start=ints(st), positions=ints(pos) if given else None)
    else:  # keys and values alone
        block = B.block(st[-1], max(rows), max(ctx), ints(ctx), ints(st))
        B.domino_paged_append(p.cache, block, 0, None, 0, qkv, qkv.stride(0), qkv[:, hkv * D:], qkv.stride(0), norm, None, kw,
                              1e-5, table, top if rot else 0, rot, pairs, None, p.ws)
    assert p.last_status() == 0
    x = qkv.view(st[-1], hq + 2 * hkv, D)
    at = torch.tensor(pos, device="cuda")
    h = H if dt == BF else 0.0
    if hq:
        want = plain_turned(x[:, :hq], qw, 1e-5, table, at, rot, pairs, norm)
        assert bool(((q.to(O.F64) - want).abs() <= h * want.abs() * 1.01 + 64 * U * float(want.abs().max())).all())
    want = plain_turned(x[:, hq:hq + hkv], kw, 1e-5, table, at, rot, pairs, norm)
    err = 64 * U * float(want.abs().max())
    slot = torch.tensor([c + i for n, c in zip(rows, ctx) for i in range(n)], device="cuda")
    req = torch.tensor([r for r, n in enumerate(rows) for _ in range(n)], device="cuda")
    where = pages.table[req, slot // page].long()
    k, v = pages.k.view(torch.uint8) if kind == E4M3 else pages.k, pages.v.view(torch.uint8) if kind == E4M3 else pages.v
    if kind == E4M3:
        check_codes(k[where, :, slot % page], pages.k_scale[where, :, slot % page], want, err)
        c, s = P.quantise(x[:, hq + hkv:])
        assert torch.equal(v[where, :, slot % page], c) and torch.equal(pages.v_scale[where, :, slot % page], s)
    else:
        got = k[where, :, slot % page].to(O.F64)
        assert bool(((got - want).abs() <= h * want.abs() * 1.01 + err).all())
        assert torch.equal(v[where, :, slot % page], x[:, hq + hkv:])
    # Everything else stays as it was.
    free = torch.ones(k.shape[0], page, dtype=torch.bool, device="cuda")
    free[where, slot % page] = False
    for now, was in zip([pages.k, pages.v, pages.k_scale, pages.v_scale], before):
        now, was = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (now, was))
        assert torch.equal(now.transpose(1, 2)[free], was.transpose(1, 2)[free])


def test_quantised_extremes():
    """Zeros, the smallest and largest values, values at the borders of codes and scales, and vectors with an infinity or a NaN."""
    D, page = 32, 16
    tiny = 2.0 ** -133  # bf16's smallest
    rows = [torch.zeros(D), torch.full((D,), tiny), torch.full((D,), 448.0), torch.full((D,), 450.0), torch.full((D,), -3.3e38),
            torch.tensor([1e30] + [1.0] * (D - 1)), torch.tensor([2.0 ** -100, 2.0 ** -110, 2.0 ** -111] + [0.0] * (D - 3)),
            torch.tensor([448.0, 1.0625, 1.1875, 0.0009765625, 0.0029296875, 17.0, 19.0, -23.0] * 4),
            torch.tensor([float("inf")] + [1.0] * (D - 1)), torch.tensor([1.0] * (D - 1) + [float("nan")]),
            torch.tensor([57344.0] * D), torch.tensor([65536.0, -1.0] * (D // 2)), torch.tensor([-0.0, 1.0] * (D // 2)),
            torch.tensor([1.9921875 * 2.0 ** 126] * D)]
    x = torch.stack(rows).to(BF).cuda()
    n = len(rows)
    pages = P.Pages(E4M3, [n], 1, page, D, 1)
    p = layer(pages, 1, n, n, 0, norm=False)
    p.append(torch.cat([x, x, x], 1), ints([0]))
    assert p.last_status() == 0
    c, s = P.quantise(x)
    for pool, scale in ((pages.k, pages.k_scale), (pages.v, pages.v_scale)):
        got = pool.view(torch.uint8)[pages.table[0, 0].long(), 0, :n]
        assert torch.equal(scale[pages.table[0, 0].long(), 0, :n], s)
        assert torch.equal(P.dequantise(got, s).nan_to_num(7.0), P.dequantise(c, s).nan_to_num(7.0))
    # Reading back gives what the codes stand for, rounded once (to an infinity where bf16 ends).
    out = torch.zeros(1, 1, n, D, dtype=BF, device="cuda"), torch.zeros(1, 1, n, D, dtype=BF, device="cuda")
    p.read(*out, ints([n]))
    assert p.last_status() == 0
    for o in out:
        assert torch.equal(o[0, 0].nan_to_num(7.0, 8.0, 9.0), P.dequantise(c, s).to(BF).nan_to_num(7.0, 8.0, 9.0))
    assert bool(torch.isnan(out[0][0, 0, 8:10]).all())


def test_infinities_without_a_norm():
    """What does not turn stays as it is."""
    pages = P.Pages(BF, [3], 1, 16, 64, 2)
    table = rope_table(20, 32)
    p = layer(pages, 1, 3, 3, 0, rope=table, norm=False)
    x = randn(gen(1), 3, 3 * 64).to(BF)
    x[1, 64 + 50] = float("inf")
    x[2, 50] = float("-inf")
    q = p.append(x, ints([0]))
    assert torch.equal(q[:, 0, 32:], x[:, 32:64])
    assert torch.equal(pages.values("k", 0, 3)[0, :, 32:], x[:, 96:128].to(O.F64))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", ["ctx", "capacity", "q_start", "position", "page", "page_high"])
def test_append_checks_lengths_and_pages_on_the_device(kind, bad):
    """What is out of bounds is reported, nothing of the row is written, and the other requests are served."""
    pages = P.Pages(kind, [16, 16], 2, 16, 64, 3, extra_places=0)
    before = pages.k.clone().view(torch.uint8), pages.v.clone().view(torch.uint8)
    p = layer(pages, 4, 8, 4, 14, rope=rope_table(16, 64))
    ctx, st, pos = [2, 3], [0, 4, 8], [2, 3, 4, 5, 3, 4, 5, 6]
    lost = int(pages.table[1, 0])
    if bad == "ctx":
        ctx[1] = 15
    elif bad == "capacity":
        ctx[1] = 13
    elif bad == "q_start":
        st[2] = 9
    elif bad == "position":
        pos[4:] = [16] * 4
    else:
        pages.table[1, 0] = -1 if bad == "page" else pages.k.shape[0]
    p.q.fill_(7.0)
    p.append(randn(gen(8), 8, 8 * 64).to(pages.rows_type), ints(ctx), q_start=ints(st), positions=ints(pos))
    assert p.last_status() == 6
    assert p.last_status() == 0
    kept = torch.ones(pages.k.shape[0], dtype=torch.bool)
    kept[int(pages.table[0, 0])] = False
    for now, was in zip((pages.k, pages.v), before):
        assert torch.equal(now.view(torch.uint8)[kept.cuda()], was[kept.cuda()])
        assert not torch.equal(now.view(torch.uint8)[~kept.cuda()], was[~kept.cuda()])
    assert kept[lost]
    assert bool((p.q[4:] == 7.0).all()) and not bool((p.q[:4] == 7.0).any())


# ---------------------------------------------------------------------------
# Back from the pages.
# ---------------------------------------------------------------------------
READ = [
    # kind, page, first, count, hkv, D, slot_major, capacity beyond the longest
    (E4M3, 16, [0], [1], 8, 128, False, 0),
    (E4M3, 64, [0, 5, 100, 3], [400, 0, 29, 63], 2, 80, True, 3),
    (E4M3, 16, [15, 16, 17], [1, 16, 130], 1, 16, False, 5),
    (E4M3, 256, [0, 200], [1000, 300], 3, 256, False, 0),
    (BF, 32, [1, 40], [200, 77], 2, 72, True, 1),
    (F32, 16, [0, 7], [33, 95], 4, 8, False, 0),
    (F32, 128, [0] * 5, [1, 64, 65, 127, 300], 8, 128, False, 9),
    (E4M3, 32, [3, 0, 31, 64], [0, 0, 5, 0], 2, 64, False, 2),
]


@pytest.mark.parametrize("case", range(len(READ)))
def test_read(case):
    kind, page, first, count, hkv, D, slot_major, more = READ[case]
    pages = P.Pages(kind, [f + n for f, n in zip(first, count)], hkv, page, D, case, slot_major)
    cap = max(count) + more
    g = gen(case)
    shape = (len(count), cap, hkv, D) if slot_major else (len(count), hkv, cap, D)
    k, v = (randn(g, *shape).to(pages.rows_type) for _ in "kv")
    if slot_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    was = k.clone(), v.clone()
    p = layer(pages, hkv, 1, 1, max(f + n for f, n in zip(first, count)))
    p.read(k, v, ints(count), first=ints(first) if any(first) else None)
    assert p.last_status() == 0
    for which, now, old in (("k", k, was[0]), ("v", v, was[1])):
        for b, (f, n) in enumerate(zip(first, count)):
            assert torch.equal(now[b, :, :n].to(O.F64), pages.values(which, b, f + n)[:, f:])
            assert torch.equal(now[b, :, n:], old[b, :, n:])


@pytest.mark.parametrize("kind", KINDS)
def test_read_checks_ranges_and_pages_on_the_device(kind):
    pages = P.Pages(kind, [40] * 5, 2, 16, 64, 4, extra_places=0)
    p = layer(pages, 2, 1, 1, 40)
    out = [torch.full((5, 2, 40, 64), 7.0, dtype=pages.rows_type, device="cuda") for _ in "kv"]
    pages.table[3, 1] = pages.k.shape[0] + 5
    p.read(*out, ints([40, 41, -1, 40, 40]), first=ints([0, 0, 0, 0, 9]))
    assert p.last_status() == 6 and p.last_status() == 0
    for which, o in zip("kv", out):
        assert torch.equal(o[0].to(O.F64), pages.values(which, 0, 40))
        assert bool((o[[1, 2, 4]] == 7.0).all()) and bool((o[3, :, 16:32] == 7.0).all())
        pages.table[3, 1] = 0
        want = pages.values(which, 3, 40)
        assert torch.equal(o[3, :, :16].to(O.F64), want[:, :16]) and torch.equal(o[3, :, 32:].to(O.F64), want[:, 32:])


def test_unusual_codes_and_scales_read_by_their_fields():
    """All 256 codes under the lowest, the highest and ordinary scale bytes."""
    D = 256
    pages = P.Pages(E4M3, [16], 1, 16, D, 5)
    at = int(pages.table[0, 0])
    pages.k.view(torch.uint8)[at, 0] = torch.arange(256, dtype=torch.uint8, device="cuda")
    pages.v.view(torch.uint8)[at, 0] = torch.arange(256, dtype=torch.uint8, device="cuda").flip(0)
    for scale in (pages.k_scale, pages.v_scale):
        scale[at, 0] = torch.tensor([0, 1, 26, 27, 100, 120, 127, 130, 134, 135, 140, 200, 247, 250, 254, 255], dtype=torch.uint8)
    p = layer(pages, 1, 1, 1, 16)
    out = [torch.zeros(1, 1, 16, D, dtype=BF, device="cuda") for _ in "kv"]
    p.read(*out, ints([16]))
    for which, o in zip("kv", out):
        want = pages.values(which, 0, 16)[0].to(BF)
        assert torch.equal(o[0, 0].nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------
ATTN = [
    # rows, ctx, hq, hkv, D, mode, window, sinks, slot_major, page
    ([1], [0], 4, 2, 128, "causal", 0, 0, False, 16),
    ([1], [700], 8, 2, 128, "causal", 0, 0, True, 64),
    ([1, 1, 1], [127, 128, 129], 8, 1, 64, "causal", 0, 0, False, 32),
    ([1] * 5, [3000, 1, 700, 2999, 64], 32, 8, 128, "causal", 0, 0, False, 128),
    ([3, 1], [500, 90], 4, 1, 80, "causal", 100, 5, False, 16),
    ([4, 4], [900, 33], 16, 4, 128, "causal", 0, 0, False, 256),
    ([2], [250], 14, 2, 96, "full", 30, 3, True, 32),
    ([16, 16], [300, 5], 8, 2, 128, "full", 64, 4, False, 16),
    ([16], [2000], 4, 1, 128, "full", 0, 0, False, 64),
    ([17, 17, 17], [0, 33, 500], 8, 2, 128, "tree", 0, 0, False, 16),
    ([5, 0, 39], [250, 3, 10], 8, 2, 64, "tree", 100, 3, True, 64),
    ([3, 3], [40, 200], 4, 1, 64, "tree", 50, 2, False, 16),
    ([300], [0], 4, 2, 128, "causal", 0, 0, False, 128),
    ([300, 129, 1], [7, 140, 1000], 4, 2, 128, "causal", 100, 5, False, 32),
    ([257], [513], 2, 2, 64, "causal", 1, 0, False, 16),
    ([200, 31], [0, 400], 5, 1, 80, "causal", 150, 130, True, 16),
    ([6], [300], 7, 1, 96, "causal", 20, 400, False, 512),
    ([20], [150], 4, 2, 256, "causal", 40, 1, False, 16),
    ([3], [50], 4, 4, 16, "causal", 0, 0, False, 32),
    ([200], [900], 8, 1, 128, "full", 0, 0, False, 64),
    ([64, 200], [1000, 1], 16, 2, 64, "causal", 0, 0, False, 16),
    ([20, 3], [300, 5], 6, 3, 16, "causal", 0, 0, True, 16),
    ([40, 3], [100, 5], 12, 3, 48, "full", 0, 0, True, 32),
]


@pytest.mark.parametrize("kind,D", [(BF, 8), (BF, 24), (BF, 72), (BF, 104), (F32, 8), (F32, 72)])
@pytest.mark.parametrize("slot_major", [False, True])
@pytest.mark.parametrize("n", [2, 20, 90])
def test_heads_of_odd_sizes(kind, D, slot_major, n):
    """Strides that are odd multiples of 16 bytes."""
    spec = ([n, n], [200, 31], 6, 3, D, "causal", 0, 0, slot_major, 16)
    check(spec, *run(kind, spec, 900 + D))


def test_layers_share_a_pool():
    """Keys and values of one allocation, several layers' pages in turn: strides beyond what a layer's own pages span."""
    g = gen(12)
    pool = randn(g, 40, 3, 2, 2, 32, 64).to(BF)  # page, layer, key or value, head, slot, element
    table = torch.randperm(40, generator=g, device="cuda").int()[:32].view(2, 16)
    for at in range(3):
        k, v = pool[:, at, 0], pool[:, at, 1]
        for n in (1, 9, 60):
            q = randn(g, 2 * n, 8, 64).to(BF)
            out, lse = PagedAttention(k, v, table, 8, 2 * n, n, 400).attend(q, ints([400, 77]), want_lse=True)
            apart = PagedAttention(k.contiguous(), v.contiguous(), table, 8, 2 * n, n, 400)
            want, wl = apart.attend(q, ints([400, 77]), want_lse=True)
            assert torch.equal(out, want) and torch.equal(lse, wl)


def run(kind, spec, seed, poison=None, scale=None, qscale=2.0, empty_row=None, prepare=None):
    from tests.test_gpu_target import tree_mask
    rows, ctx, hq, hkv, D, mode, window, sinks, slot_major, page = spec
    g = gen(seed)
    b, st = len(rows), starts(rows)
    pages = P.Pages(kind, [r + c for r, c in zip(rows, ctx)], hkv, page, D, seed, slot_major)
    q = (qscale * randn(g, st[-1], hq, D)).to(pages.rows_type)
    mask, pos = mode, None
    if mode == "tree":
        mask, depth = tree_mask(rows, max(rows), seed, empty_row)
        pos = [c + depth[st[r] + i] for r, (n, c) in enumerate(zip(rows, ctx)) for i in range(n)]
    p = layer(pages, hq, st[-1], max(rows), max(ctx), window=window, sinks=sinks, scale=scale)
    seen = []
    for r, (n, c) in enumerate(zip(rows, ctx)):
        seen.append(torch.stack([O.seen_slots(mode, window, sinks, c, n, i, pos[st[r] + i] if pos else c + i,
                                              mask[r, i].tolist() if mode == "tree" else None) for i in range(n)])
                    if n else torch.zeros(0, c, dtype=torch.bool))
    if poison is not None:  # slots that no row of the request sees, the rest of its last page, and pages that nobody has
        mine = torch.zeros(pages.k.shape[0], page, dtype=torch.bool)
        for r, (n, c) in enumerate(zip(rows, ctx)):
            if n:
                for s in seen[r].any(0).nonzero()[:, 0].tolist():
                    mine[int(pages.table[r, s // page]), s % page] = True
        dead = ~mine.cuda()
        for pool, sc in ((pages.k, pages.k_scale), (pages.v, pages.v_scale)):
            if sc is not None:
                sc.transpose(1, 2)[dead] = 255
                pool.view(torch.uint8).transpose(1, 2)[dead] = 0x7f
            else:
                pool.transpose(1, 2)[dead] = poison
    if prepare:
        prepare(pages, q)
    args = dict(q_start=ints(st), positions=ints(pos) if pos else None, mask=mask, want_lse=True)
    out, lse = p.attend(q, ints(ctx), **args)
    first = out.clone(), lse.clone()
    out, lse = p.attend(q, ints(ctx), **args)
    assert p.last_status() == 0
    # The same call gives the same bits, whatever the splits' order.
    assert torch.equal(numbers(out), numbers(first[0])) and torch.equal(numbers(lse), numbers(first[1]))
    return q, pages, p, seen, st, out, lse


def check(spec, q, pages, p, seen, st, out, lse):
    rows, ctx, hq, hkv, D = spec[:5]
    h = H if pages.rows_type == BF else 0.0
    for r, (n, c) in enumerate(zip(rows, ctx)):
        if n == 0:
            continue
        want, wlse, absv, big = O.attention(q[st[r]:st[r + 1]], torch.nan_to_num(pages.values("k", r, c + n)),
                                            torch.nan_to_num(pages.values("v", r, c + n)), p.scale, seen[r])
        e = (D + 4) * U * big + 2.0 ** -21
        tol = (2 * e + (c + n) * U + h) * absv + 1.01 * h * want.abs() + 1e-30
        got, gl = out[st[r]:st[r + 1]].to(O.F64), lse[st[r]:st[r + 1]].to(O.F64)
        assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())
        fine = torch.isfinite(wlse)
        assert torch.equal(torch.isfinite(gl), fine) and torch.equal(gl[~fine], wlse[~fine])
        assert bool(((gl - wlse).abs()[fine] <= (2 * e + (c + n) * U) + 4 * U * wlse.abs()[fine]).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_paged_attention(kind, case):
    check(ATTN[case], *run(kind, ATTN[case], 500 + case))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", [1, 3, 4, 7, 9, 10, 11, 13, 15, 17])
def test_unseen_slots_are_not_used(kind, case):
    check(ATTN[case], *run(kind, ATTN[case], 600 + case, poison=float("nan")))


SPOTS = [([1], [500], 8, 2, 128, 16), ([4, 4], [300, 130], 4, 2, 64, 64), ([16], [700], 8, 2, 128, 32),
         ([17, 17], [140, 300], 8, 2, 80, 16), ([200], [150], 8, 2, 128, 128)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spot", range(len(SPOTS)))
def test_non_finite_values_reach_only_the_rows_that_see_them(kind, spot):
    """A value of NaN (a quantised one by its scale) at a slot that later rows alone see, and one that nobody's window holds."""
    rows, ctx, hq, hkv, D, page = SPOTS[spot]
    window = 60
    spec = (rows, ctx, hq, hkv, D, "causal", window, 2, False, page)
    n, c = rows[0], ctx[0]
    late, gone = c + n // 2, min(c - window - 2, 30)

    def prepare(pages, q):
        pages.put("v", 0, late, float("nan"))
        pages.put("v", 0, gone, float("nan"))

    q, pages, p, seen, st, out, lse = run(kind, spec, 700 + spot, prepare=prepare)
    hit = seen[0][:, late].cuda()
    assert not bool(seen[0][:, gone].any()) and bool(hit.any())
    assert bool(torch.isnan(out[:n][hit]).all()) and not bool(torch.isnan(out[:n][~hit]).any())
    assert not bool(torch.isnan(lse).any())
    pages.put("v", 0, late, 1.0)
    pages.put("v", 0, gone, 1.0)
    keep = torch.ones(st[-1], dtype=torch.bool, device="cuda")
    keep[:n] = ~hit
    clean, _ = p.attend(q, ints(ctx), q_start=ints(st), want_lse=True)
    assert torch.equal(clean[keep], out[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spot", range(len(SPOTS)))
def test_a_nan_key_reaches_its_rows(kind, spot):
    rows, ctx, hq, hkv, D, page = SPOTS[spot]
    n, c = rows[0], ctx[0]
    late = c + n // 2
    pages = P.Pages(kind, [r + x for r, x in zip(rows, ctx)], hkv, page, D, 800 + spot)
    st = starts(rows)
    q = randn(gen(spot), st[-1], hq, D).to(pages.rows_type)
    p = layer(pages, hq, st[-1], max(rows), max(ctx))
    pages.put("k", 0, late, float("nan"))
    out, lse = p.attend(q, ints(ctx), q_start=ints(st), want_lse=True)
    hit = torch.arange(st[-1], device="cuda") >= n // 2
    hit[n:] = False
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert not bool(torch.isnan(out[~hit]).any()) and not bool(torch.isnan(lse[~hit]).any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,hq", [(3, 4), (20, 8), (150, 8)])
def test_rows_that_see_nothing(kind, n, hq):
    spec = ([n, n], [0, 50], hq, 2, 64, "tree", 1, 0, False, 16)
    q, pages, p, seen, st, out, lse = run(kind, spec, 31, empty_row=2)
    # Row 2 of the first request has no past and an empty mask row.
    assert bool((out[2] == 0).all()) and bool((lse[2] == float("-inf")).all())
    check(spec, q, pages, p, seen, st, out, lse)


@pytest.mark.parametrize("n", [1, 4, 16, 300])
def test_quantised_pages_give_what_their_values_give(n):
    """Over the cache in one piece that the pages read back as, the same formula: the outputs differ by roundings alone."""
    g = gen(n)
    rows, ctx, hq, hkv, D, page = [n, max(1, n - 3)], [260, 1000], 8, 2, 128, 32
    st = starts(rows)
    pages = P.Pages(E4M3, [r + c for r, c in zip(rows, ctx)], hkv, page, D, n)
    pages.k_scale.copy_((pages.k_scale.int() + torch.randint(-3, 4, pages.k_scale.shape, generator=g, device="cuda")).to(torch.uint8))
    pages.v_scale.copy_((pages.v_scale.int() + torch.randint(-9, 12, pages.v_scale.shape, generator=g, device="cuda")).to(torch.uint8))
    p = layer(pages, hq, st[-1], max(rows), max(ctx))
    k, v = (torch.zeros(2, hkv, 1400, D, dtype=BF, device="cuda") for _ in "kv")
    p.read(k, v, ints([r + c for r, c in zip(rows, ctx)]))
    whole = BlockAttention(k, v, hq, st[-1], max(rows), max(ctx))
    q = randn(g, st[-1], hq, D).to(BF)
    a, la = p.attend(q, ints(ctx), q_start=ints(st), want_lse=True)
    b, lb = whole.attend(q, ints(ctx), q_start=ints(st), want_lse=True)
    big = v.abs().amax().double()
    assert bool(((a.double() - b.double()).abs() <= 3 * H * big).all()) and bool(((la - lb).abs() <= 1e-4).all())
    assert float((a.double() - b.double()).norm() / b.double().norm()) < H


@pytest.mark.parametrize("kind", [E4M3, BF])
@pytest.mark.parametrize("n", [1, 16, 200])
def test_large_scales(kind, n):
    """Values above 57,344, whose scales take two factors."""
    spec = ([n], [130], 4, 2, 64, "causal", 0, 0, False, 16)

    def prepare(pages, q):
        for s in (0, 7, 90, 130):
            pages.put("v", 0, s, 1e6 * (1 + s))
            pages.put("k", 0, s, 70000.0 if s == 90 else 1e5)
        q.mul_(1e-6)

    check(spec, *run(kind, spec, 41, prepare=prepare))


def test_requests_share_pages():
    """A common beginning in the same pages, and the same request twice."""
    pages = P.Pages(E4M3, [200, 200, 200], 2, 16, 128, 9)
    pages.table[1, :8] = pages.table[0, :8]
    pages.table[2] = pages.table[0]
    q = randn(gen(9), 6, 8, 128).to(BF)
    q[4:] = q[:2]
    p = layer(pages, 8, 6, 2, 198)
    out, lse = p.attend(q, ints([198] * 3), want_lse=True)
    assert p.last_status() == 0
    assert torch.equal(out[:2], out[4:]) and torch.equal(lse[:2], lse[4:])
    seen = [torch.stack([O.seen_slots("causal", 0, 0, 198, 2, i, 198 + i) for i in range(2)])] * 3
    check(([2] * 3, [198] * 3, 8, 2, 128), q, pages, p, seen, [0, 2, 4, 6], out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 16, 200])
@pytest.mark.parametrize("bad", [-1, "high", -2 ** 31])
def test_missing_pages_are_reported(kind, n, bad):
    """The other request is served."""
    rows, ctx = [n, n], [300, 300]
    spec = (rows, ctx, 8, 2, 128, "causal", 0, 0, False, 32)
    q, pages, p, seen, st, out, lse = run(kind, spec, 21)
    want = out[n:].clone()
    pages.table[0, 3] = pages.k.shape[0] if bad == "high" else bad
    out, lse = p.attend(q, ints(ctx), q_start=ints(st), want_lse=True)
    assert p.last_status() == 6 and p.last_status() == 0
    assert torch.equal(out[n:], want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,mode,sinks", [(1, "causal", 0), (1, "causal", 5), (4, "causal", 20), (16, "full", 0), (17, "tree", 3), (200, "causal", 0),
                                          (200, "causal", 40)])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (256, 32)])
def test_pages_before_the_window_may_be_gone(kind, n, mode, sinks, D, page):
    """Their table entries are no pages any more, and nothing is reported."""
    window, ctx = 70, [500, 90, 1000]
    spec = ([n] * 3, ctx, 8, 2, D, mode, window, sinks, False, page)
    lost = []

    def prepare(pages, q):
        for r, c in enumerate(ctx):
            for j in range(pages.table.shape[1]):
                if (j + 1) * page <= c - window + 1 and j * page >= sinks:
                    pages.table[r, j] = -1 if j % 2 else 2 ** 31 - 1
                    lost.append(j)

    q, pages, p, seen, st, out, lse = run(kind, spec, 71 + n, prepare=prepare)
    assert lost
    pages.table.clamp_(min=0, max=pages.k.shape[0] - 1)
    check(spec, q, pages, p, seen, st, out, lse)


@pytest.mark.parametrize("kind", [E4M3, BF])
def test_offsets_pass_32_bits(kind):
    """A pool of more than 2^31 elements, its last pages in use."""
    D, hkv, page = 128, 8, 64
    n_pages = 2 ** 31 // (D * hkv * page) + 40
    t = torch.float8_e4m3fn if kind == E4M3 else BF
    pool = [torch.zeros(n_pages, hkv, page, D, dtype=t, device="cuda") for _ in "kv"]
    small = P.Pages(kind, [600, 600], hkv, page, D, 3)
    used = small.k.shape[0]
    scales = []
    for big, mine, sc in zip(pool, (small.k, small.v), (small.k_scale, small.v_scale)):
        big.view(torch.uint8)[-used:] = mine.view(torch.uint8)
        if sc is not None:
            s = torch.full((n_pages, hkv, page), 127, dtype=torch.uint8, device="cuda")
            s[-used:] = sc
            scales.append(s)
    table = torch.where(small.table >= 0, small.table + (n_pages - used), small.table)
    for n in (1, 16, 80):
        q = randn(gen(n), 2 * n, 32, D).to(BF)
        args = dict(k_scale=scales[0], v_scale=scales[1]) if scales else {}
        p = PagedAttention(*pool, table, 32, 2 * n, n, 500, **args)
        want = layer(small, 32, 2 * n, n, 500).attend(q, ints([500, 90]))
        assert torch.equal(p.attend(q, ints([500, 90])), want) and p.last_status() == 0
    qkv = randn(gen(4), 2, 48 * D).to(BF)
    p = PagedAttention(*pool, table, 32, 2, 1, 500, **args)
    m = layer(small, 32, 2, 1, 500)
    assert torch.equal(p.append(qkv, ints([500, 90])), m.append(qkv, ints([500, 90])))
    for big, mine in zip(pool, (small.k, small.v)):
        assert torch.equal(big.view(torch.uint8)[-used:], mine.view(torch.uint8))
    out = [[torch.zeros(2, hkv, 501, D, dtype=BF, device="cuda") for _ in "kv"] for _ in range(2)]
    p.read(*out[0], ints([501, 91]))
    m.read(*out[1], ints([501, 91]))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("n", [1, 16, 200])
def test_a_pass_together_on_another_stream_and_in_a_graph(n):
    """Append, attend and read one behind the other, eagerly on a second stream and as a graph whose lengths and table change
    between its replays."""
    g = gen(50 + n)
    b, hq, hkv, D, page = 3, 8, 2, 128, 16
    pages = P.Pages(E4M3, [600] * b, hkv, page, D, 6)
    start = [t.clone() for t in (pages.k.view(torch.uint8), pages.v.view(torch.uint8), pages.k_scale, pages.v_scale)]
    table0 = pages.table.clone()
    qkv = randn(g, b * n, (hq + 2 * hkv) * D).to(BF)
    ctx = ints([100, 0, 333])
    count = ctx + n
    p = layer(pages, hq, b * n, n, 350, rope=rope_table(700, D))
    k, v = (torch.zeros(b, hkv, 600, D, dtype=BF, device="cuda") for _ in "kv")

    def reset():
        for t, s in zip((pages.k.view(torch.uint8), pages.v.view(torch.uint8), pages.k_scale, pages.v_scale), start):
            t.copy_(s)

    def step():
        q = p.append(qkv, ctx)
        out = p.attend(q, ctx)
        p.read(k, v, count)
        return out

    want = step().clone(), k.clone()
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want[0]) and torch.equal(k, want[1])
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(k, want[1])
    reset()
    pages.table.copy_(table0[[1, 2, 0]])
    ctx.copy_(ints([7, 340, 99]))
    count.copy_(ctx + n)
    graph.replay()
    got = out.clone(), k.clone()
    reset()
    again = step()
    assert torch.equal(got[0], again) and torch.equal(got[1], k) and p.last_status() == 0
    assert not torch.equal(got[0], want[0])


def test_caches_share_a_workspace():
    """Calls over pages of all types and over a cache in one piece, one after the other on one workspace."""
    g = gen(77)
    calls = []
    ws = None
    for kind in KINDS:
        for n in (1, 16, 100):
            pages = P.Pages(kind, [700 + n] * 2, 2, 16, 128, n)
            p = layer(pages, 8, 2 * n, n, 700)
            calls.append((p, randn(g, 2 * n, 8, 128).to(pages.rows_type)))
    k = randn(g, 2, 2, 800, 128).to(BF)
    for n in (1, 16, 100):
        calls.append((BlockAttention(k, k.clone(), 8, 2 * n, n, 700), randn(g, 2 * n, 8, 128).to(BF)))
    ctx = ints([700, 333])
    want = [p.attend(q, ctx).clone() for p, q in calls]
    ws = B.workspace(max(p.ws.numel() for p, _ in calls))
    for p, _ in calls:
        p._ws = (ws.data_ptr(), ws.numel())
    for _ in range(3):
        for (p, q), w in zip(calls, want):
            assert torch.equal(p.attend(q, ctx), w)
    assert B.domino_last_status(ws) == 0


@pytest.mark.parametrize("kind", [E4M3, BF])
@pytest.mark.parametrize("b,n,ctx,hq,hkv,D,mode,window,sinks,page", [
    (96, 17, 200, 32, 8, 128, "tree", 0, 0, 16), (64, 16, 1500, 32, 8, 128, "full", 512, 4, 64),
    (70, 1, 900, 32, 8, 128, "causal", 0, 0, 32), (3, 1200, 700, 8, 2, 64, "causal", 0, 0, 128),
    (5, 500, 1000, 16, 4, 128, "causal", 300, 4, 16), (40, 4, 2700, 16, 4, 96, "causal", 0, 0, 256)])
def test_many_tiles_on_every_sm(kind, b, n, ctx, hq, hkv, D, mode, window, sinks, page):
    """Work lists that fill the GPU, against the cache in one piece on the same values."""
    g = gen(b)
    past = [(37 * r * r + 11 * r) % (ctx + 1) for r in range(b)]
    past[0] = ctx
    pages = P.Pages(kind, [c + n for c in past], hkv, page, D, b)
    q = randn(g, b * n, hq, D).to(BF)
    mask = mode
    if mode == "tree":
        mask = (torch.rand(b, n, n, generator=g, device="cuda") < 0.4).to(torch.uint8)
    p = layer(pages, hq, b * n, n, ctx, window=window, sinks=sinks)
    k, v = (torch.zeros(b, hkv, ctx + n, D, dtype=BF, device="cuda") for _ in "kv")
    p.read(k, v, ints([c + n for c in past]))
    whole = BlockAttention(k, v, hq, b * n, n, ctx, window=window, sinks=sinks)
    a, la = p.attend(q, ints(past), mask=mask, want_lse=True)
    w, lw = whole.attend(q, ints(past), mask=mask, want_lse=True)
    assert p.last_status() == 0 and whole.last_status() == 0
    # Two results that are each off by the weights' rounding (h of the values' weighted size) and the output's.
    big = float(v.abs().max())
    fine = torch.isfinite(lw)
    assert torch.equal(torch.isfinite(la), fine) and bool(((la - lw).abs()[fine] <= 1e-4).all())
    assert bool(((a.double() - w.double()).abs() <= 4 * H * big).all())
    assert float((a.double() - w.double()).norm() / w.double().norm()) < H
    first = a.clone()
    for _ in range(20):
        assert torch.equal(p.attend(q, ints(past), mask=mask), first)
