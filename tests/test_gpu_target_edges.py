"""The target-side operators where the window runs away from the slots, where kernels share a workspace, where weights or
values leave the ordinary range, and where a filter's bound lies far down the row. Tolerances are those of
test_gpu_target.py, whose derivation holds here too."""
import math

import pytest
import torch

from tests import target_oracle as O
from tests import test_gpu_target as T

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from draft_head_gb300 import binding as B
    from draft_head_gb300.target import BlockAttention, Sampler

BF, F32 = torch.bfloat16, torch.float32

# One block shape for each kernel: dtype, rows, query heads, kv heads, head size.
KERNELS = {
    "few_rows": (BF, [4, 1, 3], 8, 2, 128),
    "one_query_tile": (BF, [20, 1, 9], 8, 2, 64),
    "two_query_tiles": (BF, [150, 1, 70], 4, 2, 128),
    "wide_heads": (BF, [9, 1, 40], 4, 2, 256),
    "fp32": (F32, [9, 1, 40], 4, 2, 80),
}


def causal_at(kernel, ctx, shift, window, sinks, seed):
    """Attention of blocks whose row i is at position ctx + i + shift(i), into buffers that hold something else, and what
    the definition gives."""
    dt, rows, hq, hkv, D = KERNELS[kernel]
    g = T.gen(seed)
    st = T.starts(rows)
    k, v = T.cache_pair(g, dt, len(rows), hkv, ctx + max(rows) + 3, D)
    q = (2 * T.randn(g, st[-1], hq, D)).to(dt)
    pos = [ctx + i + shift(i) for n in rows for i in range(n)]
    p = BlockAttention(k, v, hq, st[-1], max(rows), ctx, window=window, sinks=sinks)
    p.out.fill_(7.0)
    p.lse.fill_(7.0)
    out, lse = p.attend(q, T.ints([ctx] * len(rows)), q_start=T.ints(st), positions=T.ints(pos), want_lse=True)
    assert p.last_status() == 0
    seen = [torch.stack([O.seen_slots("causal", window, sinks, ctx, n, i, pos[st[r] + i]) for i in range(n)])
            for r, n in enumerate(rows)]
    T.check_attention((dt, rows, [ctx] * len(rows), hq, hkv, D), q, k, v, p, seen, st, out, lse)
    return seen


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("ctx,window,sinks", [(10, 5, 4), (100, 64, 4), (150, 64, 200), (300, 70, 129), (127, 40, 128)])
def test_first_tokens_when_positions_run_ahead_of_the_slots(kernel, ctx, window, sinks):
    """Positions ahead of the slots by more than the window (a cache that has dropped slots): only first tokens are seen.
    Behind them, or ahead for some rows alone, the window covers part of the cache."""
    for n, shift in enumerate((lambda i: 650, lambda i: -20, lambda i: window - 1, lambda i: 650 if i % 3 else 0)):
        seen = causal_at(kernel, ctx, shift, window, sinks, 40 + n)
        assert n != 0 or all(int(s.sum(1).max()) <= sinks for s in seen)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("ctx", [0, 100, 300])
def test_rows_whose_window_lies_past_their_slots_see_nothing(kernel, ctx):
    """No first tokens, and a window that begins past the row itself: output 0 and lse -inf, for whole row tiles and for
    some of their rows."""
    for n, shift in enumerate((lambda i: 650, lambda i: 650 if i % 3 else 0, lambda i: 650 if i > 30 else 0)):
        seen = causal_at(kernel, ctx, shift, 40, 0, 50 + n)
        assert n != 0 or not any(bool(s.any()) for s in seen)


def test_kernels_share_a_workspace():
    """Calls that run on different kernels, one after another on one workspace: each leaves it ready for the next."""
    g = T.gen(60)
    calls = []
    for dt, b, rows, past, hq, hkv, D in ((F32, 1, 1, 2900, 1, 1, 80),      # its key tiles over many blocks
                                          (BF, 64, 1, 2900, 8, 8, 64),      # few rows, more tiles than SMs, each cut
                                          (BF, 3, 40, 2900, 8, 2, 128),     # one query tile
                                          (BF, 2, 1, 2900, 4, 2, 256),      # wide heads
                                          (BF, 2, 300, 2900, 8, 2, 128),    # two query tiles
                                          (BF, 1, 2, 2900, 8, 2, 128)):     # few rows, one request
        k, v = T.cache_pair(g, dt, b, hkv, past + rows, D)
        q = T.randn(g, b * rows, hq, D).to(dt)
        ctx = T.ints([past] * b)
        cache, block = B.kv_cache(k, v), B.block(b * rows, rows, past, ctx)
        calls.append((cache, block, hq, q, D ** -0.5, ctx, k, v))
    size = max(B.domino_block_attention_workspace_bytes(c[0], c[1], c[2]) for c in calls)

    def run(c, ws):
        out, lse = torch.full_like(c[3], 7.0), torch.full(c[3].shape[:2], 7.0, device="cuda")
        B.domino_block_attention(c[0], c[1], c[2], c[3], c[4], B.MASK_CAUSAL, None, 0, 0, out, lse, ws)
        return out, lse

    want = [run(c, B.workspace(size)) for c in calls]
    ws = B.workspace(size)
    n = len(calls)
    for first in range(n):
        for second in range(n):
            for x in (first, second):
                out, lse = run(calls[x], ws)
                assert torch.equal(out, want[x][0]) and torch.equal(lse, want[x][1]), (first, second, x)
    assert B.domino_last_status(ws) == 0


def far_down(V, tied, low, high, seed):
    """A row with one likely token and `tied` tokens each at `high` and at `low` nats below it (the rest masked), at random
    places, and noise that only a few tokens have."""
    g = T.gen(seed)
    at = torch.randperm(V, generator=g, device="cuda")[:2 * tied + 1]
    x = torch.full((V,), float("-inf"), device="cuda")
    x[at[0]] = 3.0
    x[at[1:tied + 1]] = 3.0 - high
    x[at[tied + 1:]] = 3.0 - low
    return x, at[1:tied + 1].sort()[0], at[tied + 1:].sort()[0]


@pytest.mark.parametrize("rows", [3, 800])
@pytest.mark.parametrize("high,low,share", [(17.0, 18.0, 0.995), (17.0, 18.0, 0.6), (20.0, 20.5, 0.98), (19.0, 21.4, 0.9),
                                            (16.0, 25.0, 0.999)])
def test_top_p_whose_bound_lies_far_down(rows, high, low, share):
    """The bound falls among equal logits far below the maximum: the tokens before it stay, no other does. Each row's noise
    would have a token drawn that does not stay, after one that does."""
    V, tied = 120000, 50000
    x, upper, lower = far_down(V, tied, low, high, 70)
    total = 1.0 + tied * (math.exp(-high) + math.exp(-low))
    top_p = torch.tensor((1.0 + share * tied * math.exp(-high)) / total, dtype=F32).item()
    stay = (top_p * total - 1.0) / math.exp(-high)  # of the upper tokens, in the order of their ids
    # Masses are good to 2^-20 of themselves (the exponential's argument, of up to 32, rounds at 2^-19 of a nat) and to 2^-22 of the whole.
    slack = 4 + tied * 2.0 ** -18 + total * 2.0 ** -22 / math.exp(-high)
    assert slack < 0.05 * tied and 0 < stay < tied
    inside, outside = int(upper[int(stay - slack)]), int(upper[min(tied - 1, int(stay + slack) + 2)])
    noise = torch.zeros(rows, V, device="cuda")
    noise[:, inside] = 60.0
    noise[0::2, lower[:5]] = 90.0
    noise[1::2, int(lower[-1])] = 90.0
    if stay + slack + 2 < tied - 1:
        noise[:, outside] = 80.0
    p = torch.full((rows,), top_p, device="cuda")
    s = Sampler(rows, V)
    tok, lp = s.sample(x.expand(rows, V).contiguous(), noise, None, None, p, want_logprob=True)
    assert s.last_status() == 0
    assert tok.tolist() == [inside] * rows
    assert bool(((lp + high + math.log(1.0 + stay * math.exp(-high))).abs() <= 1e-5).all())


@pytest.mark.parametrize("rows", [3, 800])
@pytest.mark.parametrize("top_k", [0, 60000])
@pytest.mark.parametrize("spread", [0.0, 1.4])
def test_top_p_counts_the_weight_of_a_long_tail(rows, top_k, spread):
    """150,000 tokens 22 nats down are some 1e-5 of a row together, and each less than 2^-31 of its largest weight: they
    count in what top-p takes its share of."""
    V, n = 151936, 150000
    g = T.gen(71)
    at = torch.randperm(V, generator=g, device="cuda")[:n + 1]
    x = torch.full((V,), float("-inf"), device="cuda")
    x[at[0]] = 0.0
    x[at[1:]] = -22.0 - spread * torch.rand(n, generator=g, device="cuda")
    value, order = x.to(O.F64).sort(descending=True, stable=True)
    before = (value.exp().cumsum(0) - value.exp())[:top_k or n + 1]
    total = float(before[-1] + value[len(before) - 1].exp())
    top_p = torch.tensor((1.0 + 0.5 * (total - 1.0)) / total, dtype=F32).item()
    # Masses are good to 2^-18 of themselves and to 2^-22 of the whole.
    room = 2.0 ** -22 * total + 2.0 ** -18 * (total - 1.0) + 4 * math.exp(-22.0)
    assert room < 0.2 * (total - 1.0)
    inside = order[int((before < top_p * total - room).sum()) - 1].item()
    outside = order[int((before < top_p * total + room).sum())].item()
    noise = torch.zeros(rows, V, device="cuda")
    noise[:, inside], noise[:, outside] = 60.0, 80.0
    s = Sampler(rows, V)
    tok = s.sample(x.expand(rows, V).contiguous(), noise, None, T.ints([top_k] * rows), torch.full((rows,), top_p, device="cuda"))
    assert s.last_status() == 0
    assert tok.tolist() == [inside] * rows


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_non_finite_value_reaches_rows_in_which_its_weight_vanishes(kernel, value):
    """Slots of scores so low that their weights are 0 in fp32, in key tiles that all rows see and in one that some see:
    a seen NaN or infinity still is not lost."""
    dt, _, hq, hkv, D = KERNELS[kernel]
    rows, past = {"few_rows": 4, "one_query_tile": 20, "two_query_tiles": 150}.get(kernel, 12), 400
    g = T.gen(80)
    k, v = T.cache_pair(g, dt, 1, hkv, past + rows, D)
    q = torch.ones(rows, hq, D, dtype=dt, device="cuda")
    far = ((torch.arange(past + rows, device="cuda") // 16) % 4 == 1)
    far[past + 2] = True
    k[0, :, far] = -200.0 * D ** -0.5
    p = BlockAttention(k, v, hq, rows, rows, past)
    out0, lse0 = (x.clone() for x in p.attend(q, T.ints([past]), want_lse=True))
    for slot in (85, past + 2):
        keep = v[0, 1, slot, 5].clone()
        v[0, 1, slot, 5] = value
        out, lse = p.attend(q, T.ints([past]), want_lse=True)
        v[0, 1, slot, 5] = keep
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[max(0, slot - past):, hq // hkv:, 5] = True
        assert not bool(torch.isfinite(out[hit]).any())
        assert torch.equal(out[~hit], out0[~hit]) and torch.equal(lse, lse0)
    assert p.last_status() == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_nan_score_reaches_the_log_sum(kernel):
    """A row that sees a NaN key, in a key tile of which it sees nothing else: output and lse are NaN. More requests than SMs, so that
    most have all their key tiles in one block."""
    dt, _, hq, hkv, D = KERNELS[kernel]
    rows, past, b = {"few_rows": 4, "one_query_tile": 20, "two_query_tiles": 150}.get(kernel, 12), 128, 200
    g = T.gen(81)
    k, v = T.cache_pair(g, dt, b, hkv, past + rows, D)
    q = T.randn(g, b * rows, hq, D).to(dt)
    k[:, 0, past] = float("nan")
    out, lse = BlockAttention(k, v, hq, b * rows, rows, past).attend(q, T.ints([past] * b), want_lse=True)
    G = hq // hkv
    assert bool(torch.isnan(out[:, :G]).all()) and bool(torch.isnan(lse[:, :G]).all())
    assert bool(torch.isfinite(out[:, G:]).all()) and bool(torch.isfinite(lse[:, G:]).all())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("where", ["first", "last", "all"])
def test_scores_of_minus_infinity_have_no_weight(kernel, where):
    """Whole key tiles whose seen scores are -inf: their slots count for nothing; if there are no others, as if none were seen."""
    dt, _, hq, hkv, D = KERNELS[kernel]
    rows, past = {"few_rows": 4, "one_query_tile": 20, "two_query_tiles": 150}.get(kernel, 12), 384
    g = T.gen(82)
    k, v = T.cache_pair(g, dt, 1, hkv, past + rows, D)
    q = (0.5 + torch.rand(rows, hq, D, generator=g, device="cuda")).to(dt)
    dead = torch.zeros(past + rows, dtype=torch.bool)
    dead[slice(0, 256) if where == "first" else slice(256, None) if where == "last" else slice(None)] = True
    k[0, :, dead.cuda()] = float("-inf")
    p = BlockAttention(k, v, hq, rows, rows, past)
    out, lse = p.attend(q, T.ints([past]), want_lse=True)
    seen = torch.stack([O.seen_slots("causal", 0, 0, past, rows, i, past + i) for i in range(rows)]) & ~dead
    T.check_attention((dt, [rows], [past], hq, hkv, D), q, torch.where(torch.isinf(k), torch.zeros_like(k), k), v, p, [seen], [0, rows], out, lse)


@pytest.mark.parametrize("kernel", KERNELS)
def test_scale_zero_weighs_all_seen_slots_alike(kernel):
    """Scale 0 makes every score 0, however large the products are (2^100 here)."""
    dt, _, hq, hkv, D = KERNELS[kernel]
    rows, past = {"few_rows": 4, "one_query_tile": 20, "two_query_tiles": 150}.get(kernel, 12), 200
    g = T.gen(83)
    k, v = T.cache_pair(g, dt, 1, hkv, past + rows, D)
    k *= 2.0 ** 50
    q = (2.0 ** 50 * T.randn(g, rows, hq, D)).to(dt)
    p = BlockAttention(k, v, hq, rows, rows, past, scale=0.0, window=150, sinks=3)
    out, lse = p.attend(q, T.ints([past]), want_lse=True)
    seen = torch.stack([O.seen_slots("causal", 150, 3, past, rows, i, past + i) for i in range(rows)])
    T.check_attention((dt, [rows], [past], hq, hkv, D), q, k, v, p, [seen], [0, rows], out, lse)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,V", [(3, 1003), (1, 9), (2, 60001), (700, 20011)])
def test_rows_at_any_alignment_give_the_same_draw(rows, V, dt):
    """Rows that begin and end inside 16-byte units, also where a slice is one unit or less: as when they are aligned."""
    x, gum = T.rows_of("peaked", rows, V, 90)
    x = x.to(dt)
    settings = [(0.8, 0, 1.0, 0.0), (0.7, 20, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 5000, 0.95, 0.0), (0.9, 0, 1.0, 0.05)]
    s = Sampler(rows, V, dtype=dt)
    for t, k, p, m in settings:
        a = (torch.full((rows,), t, device="cuda"), T.ints([k] * rows), torch.full((rows,), p, device="cuda"),
             torch.full((rows,), m, device="cuda"))
        want = None
        for pad, at in ((16, 0), (16, 1), (13, 3), (17, 7)):
            stride = (V + pad + 7) // 8 * 8 + (0 if at == 0 else at)
            buf = torch.full((rows, stride), float("inf"), device="cuda", dtype=dt)  # what is beside a row would win
            noise = torch.full((rows, stride), 50.0, device="cuda")
            buf[:, at:at + V], noise[:, at:at + V] = x, gum
            tok, lp = s.sample(buf[:, at:at + V], noise[:, at:at + V], *a, want_logprob=True)
            got = tok.clone(), lp.clone()
            want = got if want is None else want
            assert torch.equal(got[0], want[0])
            # The order of a sum's terms goes with the alignment.
            assert bool(((got[1] - want[1]).abs() <= 1e-5).all())
    assert s.last_status() == 0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bad", ["past", "negative past", "fewer rows than none", "past the cache"])
def test_lengths_of_requests_without_rows_are_reported(bad, many):
    """A bad length of a request that none of the rows leads to is reported by both calls; the rows of the others are served."""
    n, D = (3000 if many else 4), 64
    g = T.gen(95)
    k, v = T.cache_pair(g, BF, 3, 2, n + 16, D)
    ctx, st = [2, 5, 3], [0, n, n, 2 * n]
    if bad == "past":
        ctx[1] = 17
    elif bad == "negative past":
        ctx[1] = -1
    elif bad == "past the cache":
        ctx[1] = n + 17
    else:
        st = [0, n, n - 2, 2 * n - 2]
    p = BlockAttention(k, v, 4, 2 * n, n, 16)
    qkv = T.randn(g, 2 * n, 8 * D).to(BF)
    k0 = k.clone()
    q = p.append(qkv, T.ints(ctx), q_start=T.ints(st))
    assert p.last_status() == 6
    assert not torch.equal(k[0, :, 2:n], k0[0, :, 2:n]) and not torch.equal(k[2], k0[2])
    p.attend(q, T.ints(ctx), q_start=T.ints(st))
    assert p.last_status() == 6 and p.last_status() == 0
    good = [0, n, n, 2 * n]
    p.append(qkv, T.ints([2, 5, 3]), q_start=T.ints(good))
    assert p.last_status() == 0


@pytest.mark.parametrize("case", [(F32, 3, 2400, 14, 2, 80, 40, False, True), (F32, 5, 1500, 4, 4, 256, 256, False, False),
                                  (F32, 2, 3000, 8, 2, 64, 64, True, False), (F32, 4, 1500, 6, 3, 48, 20, False, True)])
def test_norm_rope_of_many_fp32_rows(monkeypatch, case):
    """As many rows as take the kernel for many in fp32 too."""
    monkeypatch.setattr(T, "MANY", [case])
    T.test_norm_rope_of_many_rows(0)


@pytest.mark.parametrize("D", [8, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 1), (3, 10, 2), (1, 2, 2), (4, 8, 2)])
def test_few_rows_in_pieces_at_every_head_size(D, rows, hq, hkv):
    """Long caches, whose row tiles are cut: the pieces' rows lie behind one another in the workspace and keep to their place,
    and to the workspace."""
    g = T.gen(96)
    ctx = [2700, 900]
    k, v = T.cache_pair(g, BF, 2, hkv, max(ctx) + rows, D)
    q = (2 * T.randn(g, 2 * rows, hq, D)).to(BF)
    p = BlockAttention(k, v, hq, 2 * rows, rows, max(ctx))
    n = p.ws.numel()
    ws = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    ws[:n] = 0
    out, lse = torch.empty_like(q), torch.empty(2 * rows, hq, device="cuda")
    past = T.ints(ctx)
    block = B.block(2 * rows, rows, max(ctx), past)
    first = None
    for _ in range(20):
        B.domino_block_attention(p.cache, block, hq, q, p.scale, B.MASK_CAUSAL, None, 0, 0, out, lse, ws[:n])
        first = first or (out.clone(), lse.clone())
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert bool((ws[n:] == 0x5a).all()) and B.domino_last_status(ws[:n]) == 0
    seen = [torch.stack([O.seen_slots("causal", 0, 0, c, rows, i, c + i) for i in range(rows)]) for c in ctx]
    T.check_attention((BF, [rows] * 2, ctx, hq, hkv, D), q, k, v, p, seen, [0, rows, 2 * rows], out, lse)
