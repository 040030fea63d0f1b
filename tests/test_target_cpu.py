"""Host-side refusals of the target-side operators (no GPU: every call is
rejected, or is a no-op, before anything is enqueued), and the 64-bit plain
forms the GPU tests compare with against library routines and closed forms."""
import ctypes
import math

import pytest
import torch

from tests import target_oracle as O

F = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def B():
    from draft_head_gb300 import build
    build.build()
    from draft_head_gb300 import binding
    return binding


def cache(B, dtype=1, batch=2, hkv=2, dim=128, cap=64, k=F, v=F, strides=None):
    rs, hs, ss = strides or (hkv * cap * dim, cap * dim, dim)
    return B.domino_kv_cache(dtype, batch, hkv, dim, cap, k, v, rs, hs, ss)


def rows(B, tokens=8, max_q=4, max_ctx=60, q_start=F, ctx=F, pos=None):
    return B.domino_block(tokens, max_q, max_ctx, q_start, ctx, pos)


def rope(B, c, r, hq=4, q=F, qs=512, k=F, ks=256, v=F, vs=256, qw=None, kw=None, eps=1e-6, table=F, max_pos=64, rot=128, q_out=F,
         ws=F, n=256):
    return B.lib.domino_qk_norm_rope(ctypes.byref(c) if c else None, ctypes.byref(r) if r else None, hq, q, qs, k, ks, v, vs, qw,
                                     kw, eps, table, max_pos, rot, 0, q_out, ws, n, None)


def attn(B, c, r, hq=4, q=F, scale=0.1, mode=0, mask=None, window=0, sinks=0, out=F, ws=F, n=1 << 40):
    return B.lib.domino_block_attention(ctypes.byref(c) if c else None, ctypes.byref(r) if r else None, hq, q, scale, mode, mask,
                                        window, sinks, out, None, ws, n, None)


BAD_CACHE = [(dict(dtype=2), 1), (dict(batch=-1), 1), (dict(hkv=0), 1), (dict(dim=0), 1), (dict(cap=0), 1), (dict(k=None), 1),
             (dict(v=F + 8), 1), (dict(strides=(4, 128, 128)), 1), (dict(strides=(-8, 128, 128)), 1),
             (dict(dim=264, strides=(0, 0, 0)), 2), (dict(dim=100, strides=(0, 0, 0)), 2), (dict(batch=65536), 2)]
BAD_ROWS = [dict(tokens=-1), dict(max_q=-1), dict(max_ctx=-1), dict(max_q=3), dict(ctx=None), dict(q_start=None, max_q=5)]


@pytest.mark.parametrize("i", range(len(BAD_CACHE)))
def test_caches_that_are_refused(B, i):
    kw, status = BAD_CACHE[i]
    assert rope(B, cache(B, **kw), rows(B), rot=0) == status
    assert attn(B, cache(B, **kw), rows(B)) == status


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_blocks_that_are_refused(B, i):
    assert rope(B, cache(B), rows(B, **BAD_ROWS[i])) == 1
    assert attn(B, cache(B), rows(B, **BAD_ROWS[i])) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(hq=-4), 1), (dict(hq=3), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(rot=3), 1), (dict(rot=130), 1),
    (dict(rot=-2), 1), (dict(table=None), 1), (dict(max_pos=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=F + 2), 1),
    (dict(qs=514), 1), (dict(ks=-8), 1), (dict(qw=F + 4), 1), (dict(q_out=None), 1), (dict(ws=None), 5), (dict(ws=F + 16), 5),
    (dict(n=255), 5)])
def test_norm_rope_refusals(B, kw, status):
    assert rope(B, cache(B), rows(B), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), 1), (dict(hq=3), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(mode=3), 1),
    (dict(mode=-1), 1), (dict(mode=2), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(q=None), 1), (dict(q=F + 8), 1),
    (dict(out=None), 1), (dict(ws=None), 5), (dict(n=256), 5)])
def test_attention_refusals(B, kw, status):
    assert attn(B, cache(B), rows(B), **kw) == status


def test_nothing_to_do_is_no_error(B):
    empty = rows(B, tokens=0, max_q=0)
    assert rope(B, cache(B), empty, k=None, v=None, q=None, ws=None, n=0) == 0
    assert attn(B, cache(B), empty, q=None, out=None, ws=None, n=0) == 0
    assert rope(B, cache(B, batch=0), empty) == 0
    assert B.lib.domino_sample(0, None, 0, 0, 5, *[None] * 5, 0, None, None, None, 0, None) == 0
    assert rope(B, None, rows(B)) == 1 and attn(B, cache(B), None) == 1


def test_attention_workspace_grows_with_no_smaller_block(B):
    size = lambda c, r, hq: B.lib.domino_block_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(r), hq)
    big = size(cache(B, batch=64, cap=9000), rows(B, tokens=64 * 16, max_q=16, max_ctx=8000), 8)
    assert big % 256 == 0 and big >= 256
    for tokens, mq, ctx in ((1, 1, 0), (64, 1, 8000), (128, 2, 100), (17, 17, 8000), (1024, 16, 8000)):
        assert size(cache(B, batch=64, cap=9000), rows(B, tokens=tokens, max_q=mq, max_ctx=ctx), 8) <= big
    assert size(cache(B, dim=100, strides=(0, 0, 0)), rows(B), 8) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(V=0), 1), (dict(logits=None), 1), (dict(logits=F + 2), 1), (dict(g=F + 2), 1),
    (dict(tokens=None), 1), (dict(g=None), 1), (dict(ls=99), 1), (dict(gs=99), 1), (dict(ws=None), 5), (dict(n=128), 5)])
def test_sample_refusals(B, kw, status):
    a = dict(dtype=0, logits=F, ls=100, rows=3, V=100, g=F, gs=100, tokens=F, ws=F, n=256)
    a.update(kw)
    assert B.lib.domino_sample(a["dtype"], a["logits"], a["ls"], a["rows"], a["V"], None, None, None, None, a["g"], a["gs"],
                               a["tokens"], None, a["ws"], a["n"], None) == status


def test_cache_struct_from_tensors(B):
    k = torch.zeros(2, 10, 3, 64, dtype=torch.bfloat16).transpose(1, 2)
    c = B.kv_cache(k, k.clone(memory_format=torch.preserve_format))
    assert (c.batch, c.n_kv_heads, c.capacity, c.head_dim) == (2, 3, 10, 64)
    assert (c.request_stride, c.head_stride, c.slot_stride) == (1920, 64, 192)
    for bad in ((k, k.contiguous()), (k.half(), k.half()), (k.float(), k), (k[..., ::2], k[..., ::2])):
        with pytest.raises(ValueError):
            B.kv_cache(*bad)


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------
def test_plain_attention_is_torch_attention():
    torch.manual_seed(0)
    q, k, v = torch.randn(5, 4, 16, dtype=O.F64), torch.randn(2, 12, 16, dtype=O.F64), torch.randn(2, 12, 16, dtype=O.F64)
    seen = torch.stack([O.seen_slots("causal", 4, 2, 7, 5, i, 7 + i) for i in range(5)])
    out, lse, _, _ = O.attention(q, k, v, 0.25, seen)
    kk, vv = k.repeat_interleave(2, 0), v.repeat_interleave(2, 0)
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=seen, scale=0.25)
    assert torch.allclose(out, want.transpose(0, 1), atol=1e-12)
    # All scores 0: the log of the number of seen slots.
    _, lse, _, _ = O.attention(q * 0, k, v, 0.25, seen)
    assert torch.allclose(lse, seen.sum(1).double().log()[:, None].expand(-1, 4))


def test_plain_visibility_hand_cases():
    assert O.seen_slots("causal", 3, 1, 5, 2, 1, 6).tolist() == [True, False, False, False, True, True, True]
    assert O.seen_slots("causal", 0, 0, 2, 3, 1, 3).tolist() == [True, True, True, True, False]
    assert O.seen_slots("full", 2, 0, 3, 2, 0, 3).tolist() == [False, False, True, True, True]
    assert O.seen_slots("tree", 1, 0, 2, 3, 2, 3, [1, 0, 1]).tolist() == [False, False, True, False, True]


def test_plain_rope_keeps_norms_and_relative_positions():
    torch.manual_seed(1)
    f = 1e4 ** (-torch.arange(0, 8, 2, dtype=O.F64) / 8)
    a = torch.arange(40, dtype=O.F64)[:, None] * f
    table = torch.cat([a.cos(), a.sin()], 1)
    x, y = torch.randn(1, 1, 8, dtype=O.F64), torch.randn(1, 1, 8, dtype=O.F64)
    for pairs in (False, True):
        at = lambda z, p: O.norm_rope(z, None, 0.0, table, torch.tensor([p]), 8, pairs)
        assert abs(float(at(x, 9).square().mean()) - 1) < 1e-12
        assert abs(float((at(x, 3) * at(y, 10)).sum() - (at(x, 20) * at(y, 27)).sum())) < 1e-9


def test_plain_draw_hand_cases():
    x = torch.tensor([0.0, 3.0, 3.0, 1.0, 2.0])
    g = torch.tensor([9.0, 0.0, 0.1, 9.0, 0.0])
    assert O.sample(x, g, 1.0, 2, 1.0, 0.0)[0] == 2
    assert O.sample(x, g, 1.0, 1, 1.0, 0.0)[:2] == (1, 0.0)
    assert O.sample(x, g, 0.0, 0, 1.0, 0.0)[:2] == (1, 0.0)
    assert O.sample(x, g, 1.0, 0, 1.0, 0.0)[0] == 3  # 1 + 9 beats 0 + 9
    assert O.sample(x, g, 1.0, 0, 0.3, 0.0)[0] == 1
    assert O.sample(x, g, 1.0, 0, 1.0, 0.5)[0] == 2
    t, lp, _ = O.sample(x, g, 1.0, 3, 1.0, 0.0)
    assert t == 2 and abs(lp + math.log(2 + math.exp(-1))) < 1e-12
