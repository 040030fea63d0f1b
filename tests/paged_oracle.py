"""Plain 64-bit forms of the operators on a cache in pages and of the token scores, from their definitions (torch float64; no
framework code), and what tests need to lay pages out."""
from __future__ import annotations

import random

import torch

F64 = torch.float64


def pow2(e):
    """2^e in float64, exact by its fields (a device's pow need not be)."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def code_values(device="cpu"):
    """The 256 e4m3 codes' values by their fields: sign, 4 bits of exponent (bias 7), 3 of mantissa; every code a number."""
    c = torch.arange(256, device=device)
    e, m = (c >> 3) & 15, (c & 7).to(F64)
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * pow2(e - 7))
    return torch.where(c >= 128, -v, v)


def dequantise(codes, scale):
    """codes [..., D] float8_e4m3fn or uint8, scale [...] uint8 -> float64."""
    s = scale.to(torch.int32)
    f = torch.where(s == 255, torch.full_like(s, float("nan"), dtype=F64), pow2(s - 127))
    return code_values(codes.device)[codes.view(torch.uint8).long()] * f[..., None]


def scale_exponent(most: float) -> int:
    e = -100
    while e < 120 and most > 448 * 2.0 ** e:
        e += 1
    return e


def quantise(x):
    """Vectors [..., D] -> (codes as uint8, scale bytes), by a search through the codes."""
    x = x.to(F64)
    flat = x.reshape(-1, x.shape[-1])
    fine = torch.isfinite(flat).all(1)
    flat = torch.where(fine[:, None], flat, torch.zeros_like(flat))
    e = torch.tensor([scale_exponent(m) for m in flat.abs().amax(1).tolist()], dtype=torch.int32, device=x.device)
    y = flat / pow2(e)[:, None]
    grid = code_values(x.device)[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    at = torch.bucketize(y.abs(), mid)
    up = (at < 126) & (y.abs() == mid[at.clamp(max=125)]) & (at % 2 == 1)
    codes = (at + up).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 7)
    codes = torch.where(fine[:, None], codes, torch.zeros_like(codes))
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return codes.reshape(x.shape), scale.reshape(x.shape[:-1])


class Pages:
    """A pool of pages [n_pages, hkv, page, D] of `kind` ("e4m3", torch.bfloat16 or torch.float32) and a table for requests of
    `slots` slots each, in random order, with a few pages that nobody has; what lies behind a request's pages is -1."""

    def __init__(self, kind, slots, hkv, page, D, seed=0, slot_major=False, device="cuda", spare=3, extra_places=1):
        self.kind, self.page, self.slots = kind, page, slots
        need = [(n + page - 1) // page for n in slots]
        total = sum(need) + spare
        order = list(range(total))
        random.Random(seed).shuffle(order)
        table, at = [], 0
        most = max(need + [1]) + extra_places
        for n in need:
            table.append(order[at:at + n] + [-1] * (most - n))
            at += n
        self.table = torch.tensor(table, dtype=torch.int32, device=device)
        g = torch.Generator(device=device)
        g.manual_seed(seed + 77)
        self.k, self.v = (self._pool(torch.randn(total, hkv, page, D, generator=g, device=device), slot_major) for _ in "kv")
        self.k_scale = self.v_scale = None
        if kind == "e4m3":
            (self.k, self.k_scale), (self.v, self.v_scale) = self.k, self.v

    def _pool(self, x, slot_major):
        if self.kind == "e4m3":
            c, s = quantise(x)
            if slot_major:
                c = c.transpose(1, 2).contiguous().transpose(1, 2)
            return c.view(torch.float8_e4m3fn), s
        x = x.to(self.kind)
        return x.transpose(1, 2).contiguous().transpose(1, 2) if slot_major else x

    @property
    def rows_type(self):
        return torch.bfloat16 if self.kind == "e4m3" else self.kind

    def values(self, which, b, n):
        """The first n slots of request b, [hkv, n, D] in float64."""
        if n == 0:
            pool = self.k
            return torch.zeros(pool.shape[1], 0, pool.shape[3], dtype=F64, device=pool.device)
        ids = self.table[b, :(n + self.page - 1) // self.page].long()
        pool, scale = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        x = dequantise(pool.view(torch.uint8)[ids], scale[ids]) if self.kind == "e4m3" else pool[ids].to(F64)
        return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]

    def put(self, which, b, s, value):
        """Slot s of request b, all heads, becomes `value` (a number, or [hkv, D]); NaN by the scale where it is quantised."""
        page, at = int(self.table[b, s // self.page]), s % self.page
        pool, scale = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        if self.kind != "e4m3":
            pool[page, :, at] = value
            return
        x = torch.as_tensor(value, dtype=F64, device=pool.device).expand(pool.shape[1], pool.shape[3])
        c, e = quantise(x)
        pool.view(torch.uint8)[page, :, at], scale[page, :, at] = c, e


def scores(logits, token, T, top_n):
    """One row: (logprob, rank, entropy, lse, ids, their log-probabilities), in 64 bits."""
    x = logits.to(F64)
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    top = float(x.max())
    if top == float("-inf"):
        lse, lp = top, torch.full_like(x, float("-inf"))
        entropy = 0.0
    else:
        d = torch.where(x == top, torch.zeros_like(x), (x - top) / T)
        w = d.exp()
        S = float(w.sum())
        lse = top / T + float(torch.log(w.sum()))
        lp = d - torch.log(w.sum())
        p = w / S
        entropy = float(-(torch.where(p > 0, p * lp, torch.zeros_like(p))).sum())
    order = torch.sort(x, descending=True, stable=True)[1]
    listed = order[:top_n][x[order[:top_n]] > float("-inf")]
    ids = torch.full((top_n,), -1, dtype=torch.int32, device=x.device)
    lps = torch.full((top_n,), float("-inf"), dtype=F64, device=x.device)
    ids[:len(listed)], lps[:len(listed)] = listed.int(), lp[listed]
    if token < 0:
        return 0.0, 0, entropy, lse, ids, lps
    return float(lp[token]), int((order == token).nonzero()[0, 0]), entropy, lse, ids, lps
