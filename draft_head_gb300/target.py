"""The target's side of a cycle: one attention layer's cache with the calls that
fill and read it for a drafted block, in one piece per request (BlockAttention) or
in pages (PagedAttention), the draw from the target's logits (Sampler) and what they
say of given tokens (TokenScorer). Buffer ownership and argument marshalling only; every
computation runs in libdomino's kernels.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding as B

_MODES = {"causal": B.MASK_CAUSAL, "full": B.MASK_FULL}


def _need(t, dtype, count: int, device: int, what: str):
    """A device array that the library takes by its address: `count` elements at least, one behind the other."""
    if t.dtype is not dtype or t.numel() < count or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: {count} elements of {dtype} on device {device}, contiguous; not {tuple(t.shape)} of {t.dtype} "
                         f"on {t.device}")


def _stream(ordinal: int):
    """torch's current stream's handle, or None where the arrays' device is not the current one: the caller goes there and asks
    again."""
    at = torch.cuda.current_device()
    if at != ordinal:
        return None
    return B._raw_stream(at) if B._raw_stream is not None else B._stream(None)


def rope_table(positions: int, rot_dim: int, base: float = 1e6, device="cuda") -> torch.Tensor:
    """The rotation table domino_qk_norm_rope reads, [positions, rot_dim] fp32: the cosines of pos * base^(-2j / rot_dim)
    for j < rot_dim / 2, then the sines (angles in 64 bits)."""
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


class _Attention:
    """What the layers share: buffers, the checks of a call's arrays, and the calls. `lib`: the library's functions that append and
    attend, by name; `norm`: arguments of the first one in front of the weights."""

    def _set_up(self, cache, device, dtype, lib, n_q_heads, max_tokens, max_q, max_ctx, window, sinks, scale, rope, q_weight, k_weight,
                eps, interleaved, norm=()):
        self.cache = cache
        self.hq, self.hkv, self.dim = n_q_heads, self.cache.n_kv_heads, self.cache.head_dim
        self.dev, self.dtype = device, dtype
        self.ordinal = device.index if device.type == "cuda" else -1
        self.max_tokens, self.max_q, self.max_ctx = max_tokens, max_q, max_ctx
        self.window, self.sinks = window, sinks
        self.scale = float(self.dim ** -0.5 if scale is None else scale)
        for weight, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if weight is not None:
                _need(weight, self.dtype, self.dim, self.ordinal, what)
        if rope is not None:
            if rope.dim() != 2:
                raise ValueError(f"rope: [positions, rot_dim], not {tuple(rope.shape)}")
            _need(rope, torch.float32, 0, self.ordinal, "rope")
        self.rope, self.q_weight, self.k_weight = rope, q_weight, k_weight
        self.eps, self.interleaved = float(eps), int(interleaved)
        self._append, self._attend = lib
        self.rows = B.block(max_tokens, max_q, max_ctx, None)
        self.ws = B.workspace(getattr(B, self._attend + "_workspace_bytes")(self.cache, self.rows, n_q_heads), self.dev)
        self.q = torch.empty(max_tokens, n_q_heads, self.dim, dtype=self.dtype, device=self.dev)
        self.out = torch.empty_like(self.q)
        self.lse = torch.empty(max_tokens, n_q_heads, dtype=torch.float32, device=self.dev)
        # Arguments that stay the same from call to call, marshalled once.
        self._refs = (ctypes.byref(self.cache), ctypes.byref(self.rows))
        self._ws = (self.ws.data_ptr(), self.ws.numel())
        self._norm = (*norm, B._ptr(q_weight), B._ptr(k_weight), self.eps, B._ptr(rope), 0 if rope is None else rope.shape[0],
                      0 if rope is None else rope.shape[1], self.interleaved, self.q.data_ptr(), *self._ws)
        self._out = (self.out.data_ptr(), self.lse.data_ptr())
        self._calls = (getattr(B.lib, self._append), getattr(B.lib, self._attend))

    def _set_rows(self, tokens: int, ctx_len, q_start, positions):
        if tokens > self.max_tokens:
            raise ValueError(f"{tokens} rows: made for {self.max_tokens}")
        r, batch, ordinal = self.rows, self.cache.batch, self.ordinal
        _need(ctx_len, torch.int32, batch, ordinal, "ctx_len")
        if q_start is not None:
            _need(q_start, torch.int32, batch + 1, ordinal, "q_start")
        if positions is not None:
            _need(positions, torch.int32, tokens, ordinal, "positions")
        r.tokens = tokens
        r.max_q = self.max_q if q_start is not None else tokens // batch
        r.ctx_len = ctx_len.data_ptr()
        r.q_start = None if q_start is None else q_start.data_ptr()
        r.positions = None if positions is None else positions.data_ptr()

    def append(self, qkv, ctx_len, q_start=None, positions=None):
        """qkv [tokens, (n_q_heads + 2 n_kv_heads) * head_dim], the projection's rows (q, k, v heads in that order):
        normed and rotated queries come back [tokens, n_q_heads, head_dim] (a buffer of this object), keys and values go
        to the cache at slots ctx_len[b] + row."""
        width = (self.hq + 2 * self.hkv) * self.dim
        if (qkv.dtype != self.dtype or qkv.dim() != 2 or qkv.shape[1] != width or qkv.stride(1) != 1 or
                qkv.get_device() != self.ordinal):
            raise ValueError(f"qkv: [tokens, {width}] of {self.dtype} on {self.dev}")
        tokens = qkv.shape[0]
        self._set_rows(tokens, ctx_len, q_start, positions)
        stream = _stream(self.ordinal)
        if stream is None:
            with torch.cuda.device(self.ordinal):
                return self.append(qkv, ctx_len, q_start, positions)
        p, stride, size = qkv.data_ptr(), qkv.stride(0), qkv.element_size()
        k = p + self.hq * self.dim * size
        st = self._calls[0](*self._refs, self.hq, p, stride, k, stride, k + self.hkv * self.dim * size, stride, *self._norm, stream)
        if st:
            raise B.DominoError(st, self._append)
        return self.q if tokens == self.max_tokens else self.q[:tokens]

    def attend(self, q, ctx_len, q_start=None, positions=None, mask="causal", want_lse: bool = False):
        """Attention of q [tokens, n_q_heads, head_dim] over the cache (the block's own keys and values are in it):
        mask "causal", "full", or a tree's [batch, max_q, max_q] uint8 (dominotree_verify's). Returns the output
        [tokens, n_q_heads, head_dim], and with want_lse the rows' log-sum-exp [tokens, n_q_heads] (buffers of this
        object)."""
        tokens = q.shape[0]
        if (q.dtype != self.dtype or q.shape[1:] != self.q.shape[1:] or not q.is_contiguous() or
                q.get_device() != self.ordinal):
            raise ValueError(f"q: [tokens, {self.hq}, {self.dim}] of {self.dtype} on {self.dev}, contiguous")
        self._set_rows(tokens, ctx_len, q_start, positions)
        if isinstance(mask, str):
            mode, mask_ptr = _MODES[mask], None
        else:
            mode, mask_ptr = B.MASK_TREE, mask.data_ptr()
            n, batch = self.rows.max_q, self.cache.batch
            if mask.dim() == 0 or mask.shape[-1] != n:
                raise ValueError(f"mask: [{batch}, {n}, {n}], not {tuple(mask.shape)}")
            _need(mask, torch.uint8, batch * n * n, self.ordinal, "mask")
        stream = _stream(self.ordinal)
        if stream is None:
            with torch.cuda.device(self.ordinal):
                return self.attend(q, ctx_len, q_start, positions, mask, want_lse)
        st = self._calls[1](*self._refs, self.hq, q.data_ptr(), self.scale, mode, mask_ptr, self.window, self.sinks, self._out[0],
                            self._out[1] if want_lse else None, *self._ws, stream)
        if st:
            raise B.DominoError(st, self._attend)
        out, lse = (self.out, self.lse) if tokens == self.max_tokens else (self.out[:tokens], self.lse[:tokens])
        return (out, lse) if want_lse else out

    def last_status(self) -> int:
        return B.domino_last_status(self.ws)


class BlockAttention(_Attention):
    """One attention layer of the target (or of the draft backbone) over its cache.

    k_cache, v_cache: [batch, n_kv_heads, capacity, head_dim], bfloat16 or float32, the same strides (any order of the
    first three axes in memory), on one device with every other array of a call. max_tokens / max_q / max_ctx bound the packed rows of a call, a request's rows and its
    past. scale defaults to head_dim ** -0.5; window 0 is the whole past. rope: a rotation table [max_pos, rot_dim]
    (rope_table), float32; q_weight, k_weight: the norms' weights [head_dim], of the cache's type. Rows are packed request after request; q_start
    [batch + 1] int32 says where each begins (None: every request has max_q rows), ctx_len [batch] int32 how many slots
    are in use, positions [tokens] int32 where each row is (None: behind the past)."""

    def __init__(self, k_cache, v_cache, n_q_heads: int, max_tokens: int, max_q: int, max_ctx: int, window: int = 0,
                 sinks: int = 0, scale=None, rope=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False):
        self.k_cache, self.v_cache = k_cache, v_cache
        self._set_up(B.kv_cache(k_cache, v_cache), k_cache.device, k_cache.dtype, ("domino_qk_norm_rope", "domino_block_attention"),
                     n_q_heads, max_tokens, max_q, max_ctx, window, sinks, scale, rope, q_weight, k_weight, eps, interleaved)


class PagedAttention(_Attention):
    """The same over a cache in pages.

    k_pages, v_pages: [n_pages, n_kv_heads, page_size, head_dim], bfloat16, float32 or float8_e4m3fn, the same strides (any order
    of the first three axes in memory); page_size a power of two from 16 to 4096. float8_e4m3fn pages have k_scale and v_scale,
    [n_pages, n_kv_heads, page_size] uint8 (or float8_e8m0fnu), a power of two for each head's vector of a slot; their queries, new
    keys and values and outputs are bfloat16. page_table [batch, max_pages] int32: where slots [page_size j, page_size (j + 1)) of a
    request are, in place from call to call; entries that no slot of a call needs are not read. norm=False: keys and queries are
    rotated without a norm. The rest is as for BlockAttention."""

    def __init__(self, k_pages, v_pages, page_table, n_q_heads: int, max_tokens: int, max_q: int, max_ctx: int, k_scale=None,
                 v_scale=None, window: int = 0, sinks: int = 0, scale=None, rope=None, norm: bool = True, q_weight=None,
                 k_weight=None, eps: float = 1e-6, interleaved: bool = False):
        cache = B.paged_cache(k_pages, v_pages, page_table, k_scale, v_scale)
        self.k_pages, self.v_pages, self.page_table, self.k_scale, self.v_scale = k_pages, v_pages, page_table, k_scale, v_scale
        if not B.domino_paged_attention_workspace_bytes(cache, B.block(max_tokens, max_q, max_ctx, None), n_q_heads):
            raise ValueError(f"pages of {k_pages.shape[2]} slots, {n_q_heads} over {k_pages.shape[1]} heads of {k_pages.shape[3]}, "
                             f"{max_tokens} rows of at most {max_q} behind {max_ctx}: not supported")
        if not norm and (q_weight is not None or k_weight is not None):
            raise ValueError("q_weight, k_weight: weights of a norm")
        dtype = torch.bfloat16 if cache.dtype == B.E4M3 else k_pages.dtype
        self._set_up(cache, k_pages.device, dtype, ("domino_paged_append", "domino_paged_attention"), n_q_heads, max_tokens, max_q,
                     max_ctx, window, sinks, scale, rope, q_weight, k_weight, eps, interleaved, (int(norm),))

    def read(self, k_out, v_out, count, first=None):
        """Slots first[b] .. first[b] + count[b] - 1 of every request (first None: 0) into slots 0 .. count[b] - 1 of a cache in
        one piece: k_out, v_out [batch, n_kv_heads, capacity, head_dim] of the queries' type. count, first [batch] int32."""
        out, batch, ordinal = B.kv_cache(k_out, v_out), self.cache.batch, self.ordinal
        if (k_out.dtype != self.dtype or (out.batch, out.n_kv_heads, out.head_dim) != (batch, self.hkv, self.dim) or
                k_out.get_device() != ordinal):
            raise ValueError(f"k_out, v_out: [{batch}, {self.hkv}, capacity, {self.dim}] of {self.dtype} on {self.dev}")
        _need(count, torch.int32, batch, ordinal, "count")
        if first is not None:
            _need(first, torch.int32, batch, ordinal, "first")
        stream = _stream(ordinal)
        if stream is None:
            with torch.cuda.device(ordinal):
                return self.read(k_out, v_out, count, first)
        st = B.lib.domino_paged_read(self._refs[0], B._ptr(first), count.data_ptr(), out.capacity, ctypes.byref(out), *self._ws, stream)
        if st:
            raise B.DominoError(st, "domino_paged_read")


class Scores(NamedTuple):
    """What TokenScorer.score gives: [rows] each, top_ids and top_logprob [rows, top_n]."""
    logprob: torch.Tensor
    rank: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: torch.Tensor
    top_logprob: torch.Tensor


class TokenScorer:
    """What logits [rows, V] (bfloat16 or float32) say of given tokens: their log-probability and rank, the rows' entropy and
    log-sum-exp and the top_n (at most 32) most likely tokens. Owns the result buffers for `rows` rows."""

    def __init__(self, rows: int, V: int, dtype=torch.float32, top_n: int = 0, device="cuda"):
        if not 0 <= top_n <= 32:
            raise ValueError(f"top_n {top_n}: 0 to 32")
        self.rows, self.V, self.dtype, self.top_n = rows, V, dtype, top_n
        self.ws = B.workspace(256, device)
        f, i = dict(dtype=torch.float32, device=device), dict(dtype=torch.int32, device=device)
        self.out = Scores(torch.empty(rows, **f), torch.empty(rows, **i), torch.empty(rows, **f), torch.empty(rows, **f),
                          torch.empty(rows, top_n, **i), torch.empty(rows, top_n, **f))
        self.dev, self.ordinal = self.ws.device, self.ws.get_device()
        self._dt = {torch.bfloat16: B.BF16, torch.float32: B.F32}[dtype]
        self._args = (*(t.data_ptr() or None for t in self.out), self.ws.data_ptr(), self.ws.numel())

    def score(self, logits, tokens=None, temperature=None) -> Scores:
        """tokens [rows] int32 (-1, or None for all rows: no token, logprob 0 and rank 0), temperature [rows] fp32 (None: 1), each
        1e-30 or more. (Sampler's 0, a greedy row, is no distribution: such a row gets NaN and last_status reports it; give it the
        temperature that its log-probabilities are wanted at.) The results are buffers of this object."""
        n, ordinal = logits.shape[0], self.ordinal
        if (n > self.rows or logits.dtype != self.dtype or logits.dim() != 2 or logits.shape[1] != self.V or logits.stride(1) != 1 or
                logits.get_device() != ordinal):
            raise ValueError(f"logits: [up to {self.rows}, {self.V}] of {self.dtype} on {self.dev}")
        if tokens is not None:
            _need(tokens, torch.int32, n, ordinal, "tokens")
        if temperature is not None:
            _need(temperature, torch.float32, n, ordinal, "temperature")
        stream = _stream(ordinal)
        if stream is None:
            with torch.cuda.device(ordinal):
                return self.score(logits, tokens, temperature)
        st = B.lib.domino_token_logprobs(self._dt, logits.data_ptr(), logits.stride(0), n, self.V, B._ptr(tokens), B._ptr(temperature),
                                         self.top_n, *self._args, stream)
        if st:
            raise B.DominoError(st, "domino_token_logprobs")
        return self.out if n == self.rows else Scores(*(t[:n] for t in self.out))

    def last_status(self) -> int:
        return B.domino_last_status(self.ws)


class Sampler:
    """Draws from logits [rows, V] (bfloat16 or float32) under per-row temperature, top-k, top-p and min-p with given
    Gumbel noise; V up to 786,432. Owns the result buffers for `rows` rows."""

    def __init__(self, rows: int, V: int, dtype=torch.float32, device="cuda"):
        self.rows, self.V, self.dtype = rows, V, dtype
        self.ws = B.workspace(256, device)
        self.tokens = torch.empty(rows, dtype=torch.int32, device=device)
        self.logprob = torch.empty(rows, dtype=torch.float32, device=device)
        self.dev, self.ordinal = self.tokens.device, self.tokens.get_device()
        self._dt = {torch.bfloat16: B.BF16, torch.float32: B.F32}[dtype]
        self._ws = (self.ws.data_ptr(), self.ws.numel())
        self._out = (self.tokens.data_ptr(), self.logprob.data_ptr())

    def sample(self, logits, gumbel, temperature=None, top_k=None, top_p=None, min_p=None, want_logprob: bool = False):
        """tokens [rows] int32 (-1: no logit above -inf), and with want_logprob their log-probabilities in the kept
        distributions. gumbel [rows, V] fp32 may be None when every temperature is 0. Settings: [rows] device tensors
        (fp32; top_k int32), None: 1, off, off, off."""
        n, V, ordinal = logits.shape[0], self.V, self.ordinal
        if (n > self.rows or logits.dtype != self.dtype or logits.dim() != 2 or logits.shape[1] != V or logits.stride(1) != 1 or
                logits.get_device() != ordinal):
            raise ValueError(f"logits: [up to {self.rows}, {V}] of {self.dtype} on {self.dev}")
        if gumbel is not None and (gumbel.dtype is not torch.float32 or gumbel.dim() != 2 or gumbel.shape[0] < n or gumbel.shape[1] < V or
                                   gumbel.stride(1) != 1 or gumbel.get_device() != ordinal):
            raise ValueError(f"gumbel: [{n}, {V}] of float32 on {self.dev}, not {tuple(gumbel.shape)} of {gumbel.dtype} on {gumbel.device}")
        if temperature is not None:
            _need(temperature, torch.float32, n, ordinal, "temperature")
        if top_k is not None:
            _need(top_k, torch.int32, n, ordinal, "top_k")
        if top_p is not None:
            _need(top_p, torch.float32, n, ordinal, "top_p")
        if min_p is not None:
            _need(min_p, torch.float32, n, ordinal, "min_p")
        st = B.lib.domino_sample(self._dt, logits.data_ptr(), logits.stride(0), n, self.V, B._ptr(temperature),
                                 B._ptr(top_k), B._ptr(top_p), B._ptr(min_p), B._ptr(gumbel),
                                 0 if gumbel is None else gumbel.stride(0), self._out[0],
                                 self._out[1] if want_logprob else None, *self._ws, B._stream(None))
        if st:
            raise B.DominoError(st, "domino_sample")
        tokens, logprob = (self.tokens, self.logprob) if n == self.rows else (self.tokens[:n], self.logprob[:n])
        return (tokens, logprob) if want_logprob else tokens

    def last_status(self) -> int:
        return B.domino_last_status(self.ws)
