"""The target-side operators against their 64-bit plain forms: norm and rotation
into the cache, attention of a block over it, the draw from logits.

Tolerances, from the arithmetic (u = 2^-24 the fp32 unit, h = 2^-8 the bf16 one (8-bit significands)):
- norm and rotation: about ten fp32 roundings on the pair's magnitude, 16 u
  (|a| + |b|), and one rounding to the output type;
- attention scores: a dot product of D fp32 terms and two roundings on
  sum |q||k| scale =: big, e = (D + 4) u big + 2^-21 (exp2 and its argument);
  weights relative error 2 e (numerator and normaliser) + N u for the sums; in
  bf16 the weights' own rounding h and the output's h |out|;
- the draw: equal tokens wherever the 64-bit decision margin exceeds 1e-4 (noise
  and logits below 2^5: a score's rounding is 2^-18; masses 1e-6 relative).
"""
import math

import pytest
import torch

from tests import target_oracle as O

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8

if torch.cuda.is_available():
    from draft_head_gb300 import binding as B
    from draft_head_gb300.target import BlockAttention, Sampler, rope_table

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def cache_pair(g, dt, b, hkv, cap, D, slot_major=False, fill=None):
    out = []
    for _ in range(2):
        x = randn(g, b, cap, hkv, D) if slot_major else randn(g, b, hkv, cap, D)
        x = x.to(dt)
        if fill is not None:
            x.fill_(fill)
        out.append(x.transpose(1, 2) if slot_major else x)
    return out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return s


# ---------------------------------------------------------------------------
# Norm and rotation.
# ---------------------------------------------------------------------------
ROPE = [
    # dtype, rows per request, ctx, hq, hkv, D, rot, interleaved, slot_major, weights, positions
    (BF, [16], [5], 32, 8, 128, 128, False, False, True, False),
    (BF, [1], [0], 4, 1, 64, 64, False, True, True, False),
    (BF, [3, 0, 17, 1], [0, 9, 2, 31], 10, 2, 80, 80, False, False, True, True),
    (F32, [7, 2], [1, 40], 6, 3, 80, 40, True, True, True, False),
    (F32, [5, 5], [0, 3], 4, 4, 256, 128, False, False, False, True),
    (BF, [5], [2], 0, 2, 96, 96, True, False, True, False),
    (BF, [9, 4], [3, 3], 8, 2, 8, 0, False, False, True, False),
    (F32, [1] * 70, list(range(70)), 2, 1, 16, 12, False, False, True, False),
    (BF, [40, 1, 700], [0, 100, 7], 32, 8, 128, 64, True, False, True, True),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_qk_norm_rope(case):
    dt, rows, ctx, hq, hkv, D, rot, pairs, slot_major, weights, given = ROPE[case]
    g = gen(100 + case)
    b, st = len(rows), starts(rows)
    cap = max(r + c for r, c in zip(rows, ctx)) + 3
    k, v = cache_pair(g, dt, b, hkv, cap, D, slot_major)
    k0, v0 = k.clone(), v.clone()
    qkv = (1.7 * randn(g, st[-1], (hq + 2 * hkv) * D)).to(dt)
    table = rope_table(cap + 50, rot) if rot else None
    qw, kw = ((1 + 0.3 * randn(g, D)).to(dt), (1 + 0.3 * randn(g, D)).to(dt)) if weights else (None, None)
    pos = [c + i for n, c in zip(rows, ctx) for i in range(n)]
    if given:
        pos = [(p * 7 + 3) % (cap + 50) for p in pos]
    p = BlockAttention(k, v, hq or hkv, st[-1], max(rows), max(ctx), rope=table, q_weight=qw, k_weight=kw, eps=1e-5,
                       interleaved=pairs)
    if hq:
        q = p.append(qkv, ints(ctx), q_start=ints(st), positions=ints(pos) if given else None)
    else:  # keys and values alone
        rows_s = B.block(st[-1], max(rows), max(ctx), ints(ctx), ints(st))
        B.domino_qk_norm_rope(p.cache, rows_s, 0, None, 0, qkv, qkv.stride(0), qkv[:, hkv * D:], qkv.stride(0), None, kw,
                              1e-5, table, table.shape[0], rot, pairs, None, p.ws)
    torch.cuda.synchronize()
    assert p.last_status() == 0
    x = qkv.view(st[-1], hq + 2 * hkv, D)
    ipos = torch.tensor(pos, device="cuda")
    h = H if dt == BF else 0.0
    want_k, want_v = k0.to(O.F64), v0.to(O.F64)

    def close(got, want, mag):
        assert bool(((got.to(O.F64) - want).abs() <= h * want.abs() * 1.01 + 32 * U * mag).all())

    if hq:
        want = O.norm_rope(x[:, :hq], qw, 1e-5, table, ipos, rot, pairs)
        close(q, want, float(want.abs().max()) * 2)
    kk = O.norm_rope(x[:, hq:hq + hkv], kw, 1e-5, table, ipos, rot, pairs)
    for r, n in enumerate(rows):
        want_k[r, :, ctx[r]:ctx[r] + n] = kk[st[r]:st[r + 1]].transpose(0, 1)
        want_v[r, :, ctx[r]:ctx[r] + n] = x[st[r]:st[r + 1], hq + hkv:].to(O.F64).transpose(0, 1)
    close(k, want_k, float(want_k.abs().max()) * 2)
    assert torch.equal(v.to(O.F64), want_v)  # values move unchanged, other slots stay
    untouched = torch.ones(b, cap, dtype=torch.bool, device="cuda")
    for r, n in enumerate(rows):
        untouched[r, ctx[r]:ctx[r] + n] = False
    assert torch.equal(k.transpose(1, 2)[untouched], k0.transpose(1, 2)[untouched])


@pytest.mark.parametrize("mask,window", [("tree", 0), ("full", 90), ("causal", 0)])
def test_attention_of_short_row_tiles_again_and_again(mask, window):
    """Row tiles of one or two key tiles, several on every SM, in calls right behind one another: all of them end, and with
    the same bits."""
    g = gen(41)
    b, n, hq, hkv, D = 96, 17, 32, 8, 128
    ctx = [(37 * r) % 200 for r in range(b)]
    k, v = cache_pair(g, BF, b, hkv, 220, D)
    q = randn(g, b * n, hq, D).to(BF)
    m = (torch.rand(b, n, n, generator=g, device="cuda") < 0.4).to(torch.uint8) if mask == "tree" else None
    p = BlockAttention(k, v, hq, b * n, n, 200, window=window)
    past = ints(ctx)
    first = p.attend(q, past, mask=mask if m is None else m).clone()
    for _ in range(400):
        out = p.attend(q, past, mask=mask if m is None else m)
    torch.cuda.synchronize()
    assert p.last_status() == 0
    assert torch.equal(out, first)


MANY = [
    # dtype, requests, rows, hq, hkv, D, rot, interleaved, in place
    (BF, 3, 2000, 8, 2, 64, 64, False, False),
    (BF, 2, 1700, 5, 1, 128, 128, True, True),
    (F32, 2, 1700, 14, 2, 80, 40, False, True),
    (F32, 5, 700, 4, 4, 256, 256, False, False),
    (BF, 70, 40, 33, 3, 24, 0, False, False),
    (BF, 4, 1200, 32, 8, 128, 12, True, False),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_norm_rope_of_many_rows(case):
    """More rows than the SMs hold at once, of requests of unlike lengths, one of them empty."""
    dt, b, n, hq, hkv, D, rot, pairs, in_place = MANY[case]
    g = gen(300 + case)
    rows = [0 if r == 1 and b > 2 else max(1, n - 17 * r) for r in range(b)]
    ctx = [(5 * r) % 11 for r in range(b)]
    st, cap = starts(rows), n + 11
    k, v = cache_pair(g, dt, b, hkv, cap, D)
    want_k, want_v = k.to(O.F64), v.to(O.F64)
    q, kk, vv = ((1.7 * randn(g, st[-1], h, D)).to(dt) for h in (hq, hkv, hkv))
    table = rope_table(cap, rot) if rot else None
    qw, kw = (1 + 0.3 * randn(g, D)).to(dt), (1 + 0.3 * randn(g, D)).to(dt)
    pos = torch.tensor([c + i for m, c in zip(rows, ctx) for i in range(m)], device="cuda")
    want_q = O.norm_rope(q, qw, 1e-5, table, pos, rot, pairs)
    new_k = O.norm_rope(kk, kw, 1e-5, table, pos, rot, pairs)
    out, ws = q if in_place else torch.empty_like(q), B.workspace(256)
    block = B.block(st[-1], max(rows), max(ctx), ints(ctx), ints(st))
    B.domino_qk_norm_rope(B.kv_cache(k, v), block, hq, q, hq * D, kk, hkv * D, vv, hkv * D, qw, kw, 1e-5, table,
                          cap if rot else 0, rot, pairs, out, ws)
    assert B.domino_last_status(ws) == 0
    h = H if dt == BF else 0.0
    for r, m in enumerate(rows):
        want_k[r, :, ctx[r]:ctx[r] + m] = new_k[st[r]:st[r + 1]].transpose(0, 1)
        want_v[r, :, ctx[r]:ctx[r] + m] = vv[st[r]:st[r + 1]].to(O.F64).transpose(0, 1)
    for got, want in ((out, want_q), (k, want_k)):
        assert bool(((got.to(O.F64) - want).abs() <= h * want.abs() * 1.01 + 64 * U * float(want.abs().max())).all())
    assert torch.equal(v.to(O.F64), want_v)


def test_norm_rope_in_place_and_without_q_start():
    g = gen(7)
    k, v = cache_pair(g, BF, 3, 2, 20, 64)
    k2, v2 = k.clone(), v.clone()
    table = rope_table(20, 64)
    q, kk, vv = (randn(g, 12, n, 64).to(BF) for n in (4, 2, 2))
    ctx, ws, out = ints([0, 5, 16]), B.workspace(256), torch.empty_like(q)
    rows = B.block(12, 4, 16, ctx)
    B.domino_qk_norm_rope(B.kv_cache(k, v), rows, 4, q, 256, kk, 128, vv, 128, None, None, 1e-6, table, 20, 64, False,
                          out, ws)
    B.domino_qk_norm_rope(B.kv_cache(k2, v2), B.block(12, 4, 16, ctx, ints([0, 4, 8, 12])), 4, q, 256, kk, 128, vv, 128,
                          None, None, 1e-6, table, 20, 64, False, q, ws)
    assert B.domino_last_status(ws) == 0
    assert torch.equal(q, out) and torch.equal(k, k2) and torch.equal(v, v2)


def test_device_side_lengths_are_checked():
    """A past, a row count, a slot or a position out of its bound is reported, and nothing of the request is written; the
    other requests are served."""
    g = gen(8)
    table = rope_table(16, 64)
    for bad in ("ctx", "ctx_neg", "capacity", "q_start", "position"):
        k, v = cache_pair(g, BF, 2, 2, 16, 64)
        k0 = k.clone()
        p = BlockAttention(k, v, 4, 8, 4, 14, rope=table)
        ctx, st, pos = [2, 3], [0, 4, 8], [0, 1, 2, 3, 3, 4, 5, 6]
        if bad == "ctx":
            ctx[1] = 15
        elif bad == "ctx_neg":
            ctx[1] = -1
        elif bad == "capacity":
            ctx[1] = 14
        elif bad == "q_start":
            st[2] = 9
        else:
            pos[4:] = [16] * 4
        qkv = randn(g, 8, 8 * 64).to(BF)
        p.append(qkv, ints(ctx), q_start=ints(st), positions=ints(pos))
        assert p.last_status() == 6
        assert p.last_status() == 0
        assert torch.equal(k[1], k0[1])
        assert not torch.equal(k[0], k0[0])
        if bad != "position":
            p.out.fill_(7.0)
            p.attend(p.q, ints(ctx), q_start=ints(st))
            assert p.last_status() == 6
            assert bool((p.out[4:] == 7.0).all()) and not bool((p.out[:4] == 7.0).any())


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------
ATTN = [
    # dtype, rows, ctx, hq, hkv, D, mode, window, sinks, slot_major
    (BF, [1], [0], 4, 2, 128, "causal", 0, 0, False),
    (BF, [1], [1], 32, 8, 128, "causal", 0, 0, False),
    (BF, [1], [700], 8, 2, 128, "causal", 0, 0, True),
    (BF, [1, 1, 1], [127, 128, 129], 8, 1, 64, "causal", 0, 0, False),
    (BF, [16, 16], [300, 5], 8, 2, 128, "full", 64, 4, False),
    (BF, [16], [2000], 4, 1, 128, "full", 0, 0, False),
    (BF, [17, 17, 17], [0, 33, 500], 8, 2, 128, "tree", 0, 0, False),
    (BF, [5, 0, 39], [250, 3, 10], 8, 2, 64, "tree", 100, 3, True),
    (BF, [300], [0], 4, 2, 128, "causal", 0, 0, False),
    (BF, [300, 129, 1], [7, 140, 1000], 4, 2, 128, "causal", 100, 5, False),
    (BF, [257], [513], 2, 2, 64, "causal", 1, 0, False),
    (BF, [200, 31], [0, 400], 5, 1, 80, "causal", 150, 130, True),
    (BF, [6], [300], 7, 1, 96, "causal", 20, 400, False),
    (BF, [20], [150], 4, 2, 256, "causal", 40, 1, False),
    (BF, [3], [50], 4, 4, 8, "causal", 0, 0, False),
    (F32, [1], [1500], 4, 2, 128, "causal", 0, 0, False),
    (F32, [40, 3, 17], [3, 500, 120], 6, 2, 80, "causal", 70, 3, False),
    (F32, [9, 9], [0, 65], 4, 4, 64, "tree", 30, 2, True),
    (F32, [16], [70], 8, 1, 256, "full", 10, 1, False),
    (F32, [200], [0], 2, 1, 128, "causal", 64, 4, False),
]


def tree_mask(rows, max_q, seed, empty_row=None):
    """Random ancestor masks [batch, max_q, max_q] and depths; row `empty_row` of each sees no block row."""
    import random
    rng = random.Random(seed)
    m = torch.zeros(len(rows), max_q, max_q, dtype=torch.uint8)
    depth = []
    for b, n in enumerate(rows):
        d = [0] * n
        for i in range(n):
            if i:
                par = rng.randrange(i)
                m[b, i] = m[b, par]
                d[i] = d[par] + 1
            m[b, i, i] = 1
        if empty_row is not None and n > empty_row:
            m[b, empty_row] = 0
        depth += d
    return m.cuda(), depth


def run_attention(spec, seed, poison=None, scale=None, qscale=2.0, empty_row=None, extra=5):
    dt, rows, ctx, hq, hkv, D, mode, window, sinks, slot_major = spec
    g = gen(seed)
    b, st = len(rows), starts(rows)
    cap = max(r + c for r, c in zip(rows, ctx)) + extra
    k, v = cache_pair(g, dt, b, hkv, cap, D, slot_major)
    q = (qscale * randn(g, st[-1], hq, D)).to(dt)
    mask, pos = mode, None
    if mode == "tree":
        mask, depth = tree_mask(rows, max(rows), seed, empty_row)
        pos = [c + depth[st[r] + i] for r, (n, c) in enumerate(zip(rows, ctx)) for i in range(n)]
    p = BlockAttention(k, v, hq, st[-1], max(rows), max(ctx), window=window, sinks=sinks, scale=scale)
    seen = []
    for r, (n, c) in enumerate(zip(rows, ctx)):
        seen.append(torch.stack([O.seen_slots(mode, window, sinks, c, n, i, pos[st[r] + i] if pos else c + i,
                                              mask[r, i].tolist() if mode == "tree" else None) for i in range(n)])
                    if n else torch.zeros(0, c, dtype=torch.bool))
    if poison is not None:  # slots that no row of the request sees, and all after its rows
        for r, (n, c) in enumerate(zip(rows, ctx)):
            dead = torch.ones(cap, dtype=torch.bool)
            if n:
                dead[:c + n] = ~seen[r].any(0)
            k[r, :, dead.cuda()] = poison
            v[r, :, dead.cuda()] = poison
    out, lse = p.attend(q, ints(ctx), q_start=ints(st), positions=ints(pos) if pos else None, mask=mask, want_lse=True)
    first = out.clone(), lse.clone()
    out, lse = p.attend(q, ints(ctx), q_start=ints(st), positions=ints(pos) if pos else None, mask=mask, want_lse=True)
    torch.cuda.synchronize()
    assert p.last_status() == 0
    # The same call gives the same bits, whatever the splits' order.
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    return q, k, v, p, seen, st, out, lse


def check_attention(spec, q, k, v, p, seen, st, out, lse):
    dt, rows, ctx, hq, hkv, D = spec[:6]
    h = H if dt == BF else 0.0
    for r, (n, c) in enumerate(zip(rows, ctx)):
        if n == 0:
            continue
        want, wlse, absv, big = O.attention(q[st[r]:st[r + 1]], torch.nan_to_num(k[r, :, :c + n].float()),
                                            torch.nan_to_num(v[r, :, :c + n].float()), p.scale, seen[r])
        e = (D + 4) * U * big + 2.0 ** -21
        tol = (2 * e + (c + n) * U + h) * absv + 1.01 * h * want.abs() + 1e-30
        got, gl = out[st[r]:st[r + 1]].to(O.F64), lse[st[r]:st[r + 1]].to(O.F64)
        assert bool(torch.isfinite(got).all())
        worst = float(((got - want).abs() / tol).max())
        assert worst <= 1.0, (r, worst)
        none = torch.isinf(wlse)
        assert torch.equal(none, torch.isinf(gl)) and bool((gl[none] < 0).all())
        assert bool((got[none] == 0).all())
        assert bool(((gl - wlse)[~none].abs() <= 2 * e + (c + n) * U + 4 * U * wlse[~none].abs()).all())


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_block_attention(case):
    r = run_attention(ATTN[case], 300 + case)
    check_attention(ATTN[case], *r)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", [2, 4, 6, 7, 9, 10, 11, 16, 17])
def test_unseen_slots_are_not_used(case, poison):
    r = run_attention(ATTN[case], 400 + case, poison=poison)
    check_attention(ATTN[case], *r)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_rows_that_see_nothing(dt, D):
    """A tree row with an all-zero mask row and no past: output 0, lse -inf."""
    spec = (dt, [9, 4], [0, 0], 4, 2, D, "tree", 0, 0, False)
    r = run_attention(spec, 11, empty_row=2)
    assert bool((r[6][2] == 0).all()) and bool(torch.isneginf(r[7][2]).all())
    check_attention(spec, *r)


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 80)])
@pytest.mark.parametrize("qscale", [0.0, 40.0])
def test_flat_and_sharp_softmax(dt, D, qscale):
    """All scores equal, and scores so far apart that one key has all the weight."""
    spec = (dt, [19, 2], [400, 90], 4, 2, D, "causal", 0, 0, False)
    check_attention(spec, *run_attention(spec, 12, qscale=qscale))


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (BF, 80), (F32, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_reach_only_the_rows_that_see_them(dt, D, value):
    """A non-finite v in a slot that some rows see and others do not."""
    for spec, slot in (((dt, [12], [130], 4, 2, D, "causal", 0, 0, False), 130 + 5),
                       ((dt, [200], [30], 4, 2, D, "causal", 60, 2, False), 100),
                       ((dt, [9], [700], 4, 2, D, "tree", 0, 0, False), 700 + 3)):
        _, rows, ctx, hq, hkv, _, mode, window, sinks, _ = spec
        q, k, v, p, seen, st, out0, lse0 = run_attention(spec, 13)
        mask, pos = mode, None
        if mode == "tree":
            mask, depth = tree_mask(rows, max(rows), 13)
            pos = ints([ctx[0] + d for d in depth])
        out0, lse0 = out0.clone(), lse0.clone()
        v[0, 1, slot, 3] = value
        out, lse = p.attend(q, ints(ctx), q_start=ints(st), positions=pos, mask=mask, want_lse=True)
        hit = seen[0][:, slot].cuda()
        assert 0 < int(hit.sum()) < rows[0]
        G = hq // hkv
        assert torch.equal(lse, lse0)
        want = out0.clone()
        bad = out[hit][:, G:2 * G, 3]
        assert bool((torch.isnan(bad) if math.isnan(value) else bad == value).all())
        rest = torch.ones_like(out, dtype=torch.bool)
        rest[hit.nonzero()[:, 0], G:2 * G, 3] = False
        assert torch.equal(out[rest], want[rest])


def test_single_rows_match_the_prompt():
    """Decoding token by token over the cache gives the prompt's rows (to the output's rounding)."""
    g = gen(14)
    n, hq, hkv, D = 70, 8, 2, 128
    k, v = cache_pair(g, BF, 1, hkv, n, D)
    q = randn(g, n, hq, D).to(BF)
    whole = BlockAttention(k, v, hq, n, n, 0, window=33, sinks=2)
    one = BlockAttention(k, v, hq, 1, 1, n, window=33, sinks=2)
    a = whole.attend(q, ints([0])).float()
    for i in range(n):
        b = one.attend(q[i:i + 1], ints([i])).float()[0]
        assert float((a[i] - b).abs().max()) <= 2 * H * float(v.float().abs().max())


def test_attention_on_another_stream_and_in_a_graph():
    spec = (BF, [16, 16], [900, 40], 8, 2, 128, "full", 0, 0, False)
    q, k, v, p, seen, st, out, lse = run_attention(spec, 15)
    want = out.clone()
    ctx, qs = ints([900, 40]), ints(st)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out.zero_()
        p.attend(q, ctx, q_start=qs, mask="full")
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.attend(q, ctx, q_start=qs, mask="full")
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and p.last_status() == 0


def test_long_cache_offsets_pass_32_bits():
    """A cache whose last request's elements lie beyond 2^31 (and 2^32 bytes): bf16, 3 requests of 2^20 slots x 8 x 128."""
    g = gen(16)
    cap, hkv, D = 1 << 20, 8, 128
    k = torch.zeros(3, cap, hkv, D, dtype=BF, device="cuda").transpose(1, 2)
    v = torch.zeros(3, cap, hkv, D, dtype=BF, device="cuda").transpose(1, 2)
    ctx = cap - 10
    for x in (k, v):
        x[2, :, :64] = randn(g, hkv, 64, D).to(BF)
        x[2, :, ctx - 300:] = randn(g, hkv, 310, D).to(BF)
    spec = (BF, [4], [ctx], 16, hkv, D, "causal", 200, 8, True)
    q = randn(g, 12, 16, D).to(BF)
    p = BlockAttention(k, v, 16, 12, 4, ctx, window=200, sinks=8)
    out, lse = p.attend(q, ints([7, 9, ctx]), want_lse=True)
    assert p.last_status() == 0
    at = list(range(8)) + list(range(ctx - 300, ctx + 4))
    slots = torch.tensor(at)
    near = torch.stack([(slots < 8) | ((slots > ctx + i - 200) & (slots <= ctx + i)) for i in range(4)])
    want, wlse, absv, big = O.attention(q[8:], k[2][:, at], v[2][:, at], p.scale, near)
    e = (D + 4) * U * big + 2.0 ** -21
    assert bool(((out[8:].to(O.F64) - want).abs() <= (2 * e + 300 * U + H) * absv + 1.01 * H * want.abs()).all())
    assert bool(((lse[8:].to(O.F64) - wlse).abs() <= 2 * e + 300 * U).all())
    # The other requests' pasts are zeros: the mean of the zero values.
    assert bool((out[:8] == 0).all())


@pytest.mark.parametrize("dt,rows,ctx,hq,hkv,D,mode,window,sinks", [
    (BF, [16] * 48, [1200] * 47 + [40], 16, 4, 128, "full", 1000, 4),      # many requests: several key tiles per CTA
    (BF, [1] * 200, [300] * 200, 8, 4, 64, "causal", 0, 0),                # several row tiles per CTA
    (BF, [2500, 1300], [0, 700], 8, 4, 128, "causal", 600, 130),           # prompts, two query tiles
    (BF, [2500], [100], 8, 4, 64, "causal", 0, 0),
    (F32, [300, 40], [0, 500], 4, 2, 128, "causal", 200, 3)])
def test_many_tiles_per_cta(dt, rows, ctx, hq, hkv, D, mode, window, sinks):
    g = gen(17)
    st, cap = starts(rows), max(r + c for r, c in zip(rows, ctx))
    k, v = cache_pair(g, dt, len(rows), hkv, cap, D)
    q = (2 * randn(g, st[-1], hq, D)).to(dt)
    p = BlockAttention(k, v, hq, st[-1], max(rows), max(ctx), window=window, sinks=sinks)
    for _ in range(3):
        out, lse = p.attend(q, ints(ctx), q_start=ints(st), mask=mode, want_lse=True)
    assert p.last_status() == 0
    h = H if dt == BF else 0.0
    for r, (n, c) in enumerate(zip(rows, ctx)):
        s, i = torch.arange(c + n, device="cuda")[None], torch.arange(n, device="cuda")[:, None]
        seen = (s < sinks) | (s > c + i - window) if window else torch.ones(n, c + n, dtype=torch.bool, device="cuda")
        seen = (seen & (s <= c + i)) if mode == "causal" else seen | (s >= c)
        kk, vv = k[r, :, :c + n].to(O.F64), v[r, :, :c + n].to(O.F64)
        for hh in range(hq):
            x = q[st[r]:st[r + 1], hh].to(O.F64)
            score = torch.where(seen, (x @ kk[hh * hkv // hq].T) * p.scale, -math.inf)
            big = float((x.abs() @ kk[hh * hkv // hq].abs().T).max()) * p.scale
            w = torch.softmax(score, 1)
            e = (D + 4) * U * big + 2.0 ** -21
            want = w @ vv[hh * hkv // hq]
            tol = (2 * e + (c + n) * U + h) * (w @ vv[hh * hkv // hq].abs()) + 1.01 * h * want.abs()
            assert bool(((out[st[r]:st[r + 1], hh].to(O.F64) - want).abs() <= tol).all()), (r, hh)
            assert bool(((lse[st[r]:st[r + 1], hh].to(O.F64) - torch.logsumexp(score, 1)).abs() <= 2 * e + (c + n) * U).all())


# ---------------------------------------------------------------------------
# The draw.
# ---------------------------------------------------------------------------
def rows_of(kind, rows, V, seed):
    g = gen(seed)
    x = randn(g, rows, V)
    if kind == "peaked":
        x *= 2
        at = torch.randint(0, V, (rows, 30), generator=g, device="cuda")
        x.scatter_add_(1, at, 14 * torch.rand(rows, 30, generator=g, device="cuda"))
    elif kind == "ties":
        x = (x * 2).round() / 2
    elif kind == "equal":
        x = torch.full_like(x, 1.5)
    elif kind == "masked":  # most of the vocabulary masked, some rows to the type's lowest value
        dead = torch.rand(rows, V, generator=g, device="cuda") < 0.9
        x[dead] = float("-inf")
        x[::2][dead[::2]] = torch.finfo(torch.float32).min
        x[:, V // 2] = 0.5
    elif kind == "wide":
        x *= 1e4
    elif kind == "tiny":
        x *= 1e-30
    u = (torch.randint(0, 1 << 24, (rows, V), generator=g, device="cuda").float() + 0.5) / float(1 << 24)
    return x, -torch.log(-torch.log(u))


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.05), (0.6, 0, 0.95, 0.0), (1.0, 1, 1.0, 0.0), (0.0, 5, 0.5, 0.5),
            (1.3, 50, 1.0, 0.0), (0.9, 0, 1.0, 0.1), (1.0, 0, 1e-6, 0.0), (0.8, 1000, 0.9, 0.0), (1.0, 3000, 0.99, 1.0),
            (0.05, 0, 0.9, 0.0), (2.0, 10 ** 6, 0.5, 0.01), (1.0, 2, 0.3, 0.0), (1e-3, 40, 0.999, 0.0)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50257])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties", "equal", "masked", "wide", "tiny"])
def test_sample(kind, V, dt):
    if kind == "masked" and V < 31:
        pytest.skip("nothing to mask")
    rows = len(SETTINGS)
    x, gum = rows_of(kind, rows, V, V + len(kind))
    x = x.to(dt)
    t, k, p, m = (torch.tensor([s[j] for s in SETTINGS], device="cuda", dtype=torch.int32 if j == 1 else F32) for j in range(4))
    s = Sampler(rows, V, dtype=dt)
    tok, lp = s.sample(x, gum, t, k, p, m, want_logprob=True)
    assert s.last_status() == 0
    tok, lp = tok.tolist(), lp.tolist()
    compared = 0
    for r in range(rows):
        args = [float(y[r]) for y in (t, k, p, m)]
        want, wlp, margin = O.sample(x[r].cpu(), gum[r].cpu(), args[0], int(args[1]), args[2], args[3])
        # fp32 scores of magnitude |logit / T| round at 2^-23 of it
        bar = 1e-4 + float(x[r].float().abs().clamp(max=1e30).max()) / max(args[0], 1e-30) * 2.0 ** -22 if args[0] else 0.0
        if margin <= bar:
            continue
        compared += 1
        assert tok[r] == want, (r, margin)
        # The kept mass is off by at most what sits at the boundaries: a token there has at most its weight.
        assert lp[r] == wlp or abs(lp[r] - wlp) <= 1e-5 + 4e-6 * abs(wlp) + bar / 16, (r, lp[r], wlp)
    assert compared >= (rows // 2 if kind not in ("wide", "tiny", "masked") else 1)


def test_sample_extremes():
    V = 777
    x = torch.zeros(6, V, device="cuda")
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2, 5], x[2, 6] = float("nan"), 9.0
    x[3, 100] = x[3, 40] = float("inf")
    x[4, :] = float("-inf")
    x[4, 776] = -3.0
    x[5, :] = torch.finfo(torch.float32).min
    gum = torch.zeros(6, V, device="cuda")
    s = Sampler(6, V)
    tok, lp = s.sample(x, gum, torch.full((6,), 0.5, device="cuda"), want_logprob=True)
    assert tok.tolist() == [-1, -1, 6, 40, 776, 0]
    assert s.last_status() == 0
    lp = lp.tolist()
    assert lp[0] == lp[1] == float("-inf") and abs(lp[3] + math.log(2)) < 1e-6 and lp[4] == 0.0
    assert abs(lp[5] + math.log(V)) < 1e-5
    greedy = s.sample(x, None, torch.zeros(6, device="cuda"))
    assert greedy.tolist() == [-1, -1, 6, 40, 776, 0]


def test_sample_refuses_settings_on_the_device():
    V = 300
    x, gum = rows_of("flat", 7, V, 3)
    s = Sampler(7, V)
    t = torch.tensor([-1.0, float("nan"), 1, 1, 1, 1, 1], device="cuda")
    k = ints([0, 0, -1, 0, 0, 0, 0])
    p = torch.tensor([1, 1, 1, 0.0, 1.5, 1, 1], device="cuda")
    m = torch.tensor([0, 0, 0, 0, 0, 1.5, 0], device="cuda")
    tok, lp = s.sample(x, gum, t, k, p, m, want_logprob=True)
    assert s.last_status() == 6 and s.last_status() == 0
    assert tok.tolist()[:6] == [-1] * 6 and all(math.isnan(y) for y in lp.tolist()[:6])
    assert tok.tolist()[6] == int((x[6] + gum[6]).argmax())
    # No noise and a temperature above 0.
    s.sample(x, None, torch.ones(7, device="cuda"))
    assert s.last_status() == 6


def test_sample_strides_and_default_settings():
    x, gum = rows_of("peaked", 5, 1201, 4)
    s = Sampler(5, 1000)
    tok = s.sample(x[:, 7:1007], gum[:, 100:1100]).clone()
    want = (x[:, 7:1007] + gum[:, 100:1100]).argmax(1)
    assert tok.tolist() == want.tolist()
    one = Sampler(1, 1000)
    for r in range(5):  # a row alone gives what it gives among others
        assert one.sample(x[r:r + 1, 7:1007], gum[r:r + 1, 100:1100]).item() == tok[r].item()


@pytest.mark.parametrize("rows", [2, 200])
def test_sample_gives_the_same_bits_again(rows):
    """Candidates are gathered in whatever order the atomics take: tokens and log-probabilities do not depend on it."""
    V = 60000
    x, gum = rows_of("peaked", rows, V, 9)
    s = Sampler(rows, V)
    for k, p in ((1000, 0.99), (2000, 1.0), (300, 0.9), (0, 0.95), (64, 0.9)):
        kk, pp = ints([k] * rows), torch.full((rows,), p, device="cuda")
        first = [y.clone() for y in s.sample(x, gum, None, kk, pp, want_logprob=True)]
        for _ in range(10):
            tok, lp = s.sample(x, gum, None, kk, pp, want_logprob=True)
            assert torch.equal(tok, first[0]) and torch.equal(lp, first[1])
    assert s.last_status() == 0


@pytest.mark.parametrize("dt", [F32, BF])
def test_sample_full_vocabulary_rows(dt):
    """Long rows: filters over 151936 tokens, flat (most of the vocabulary stays) and peaked."""
    V = 151936
    for kind in ("flat", "peaked"):
        x, gum = rows_of(kind, 6, V, 5)
        x = x.to(dt)
        sets = [(1.0, 0, 0.95, 0.0), (0.7, 20, 0.8, 0.0), (1.0, 60000, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 5000, 1.0, 0.0),
                (1.0, 0, 1.0, 0.0)]
        t, k, p, m = (torch.tensor([s[j] for s in sets], device="cuda", dtype=torch.int32 if j == 1 else F32) for j in range(4))
        s = Sampler(6, V, dtype=dt)
        tok, lp = s.sample(x, gum, t, k, p, m, want_logprob=True)
        tok2, lp2 = tok.clone(), lp.clone()
        s.sample(x, gum, t, k, p, m, want_logprob=True)
        assert torch.equal(tok, tok2) and torch.equal(lp, lp2)
        for r in range(6):
            want, wlp, margin = O.sample(x[r], gum[r], *[float(t[r]), int(k[r]), float(p[r]), float(m[r])])
            if margin > 1e-4:
                assert tok[r].item() == want
                assert abs(lp[r].item() - wlp) <= 2e-5
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind,dt,rows,V", [("flat", F32, 400, 151936), ("equal", F32, 300, 151936), ("ties", BF, 300, 151936),
                                            ("masked", F32, 900, 45001), ("peaked", BF, 900, 45001), ("wide", F32, 900, 45001)])
def test_sample_of_many_rows(kind, dt, rows, V):
    """More rows than the SMs hold at once, in which a block takes a longer part of a row."""
    x, gum = rows_of(kind, rows, V, 17)
    x = x.to(dt)
    sets = [SETTINGS[r % len(SETTINGS)] for r in range(rows)]
    t, k, p, m = (torch.tensor([s[j] for s in sets], device="cuda", dtype=torch.int32 if j == 1 else F32) for j in range(4))
    s = Sampler(rows, V, dtype=dt)
    tok, lp = (y.tolist() for y in s.sample(x, gum, t, k, p, m, want_logprob=True))
    assert s.last_status() == 0
    compared = 0
    for r in range(0, rows, 7 if len(SETTINGS) % 7 else 11):
        want, wlp, margin = O.sample(x[r], gum[r], float(t[r]), int(k[r]), float(p[r]), float(m[r]))
        # As in test_sample: fp32 scores of magnitude |logit / T| round at 2^-23 of it.
        bar = 1e-4 + float(x[r].float().abs().clamp(max=1e30).max()) / max(float(t[r]), 1e-30) * 2.0 ** -22 if t[r] else 0.0
        if margin <= bar:
            continue
        compared += 1
        assert tok[r] == want, (r, margin)
        assert lp[r] == wlp or abs(lp[r] - wlp) <= 2e-5 + 4e-6 * abs(wlp) + bar / 16, (r, lp[r], wlp)
    assert compared >= 1
