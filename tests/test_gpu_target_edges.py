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
