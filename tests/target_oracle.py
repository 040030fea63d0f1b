"""Plain 64-bit forms of the target-side operators, request by request and row
by row from their definitions (torch float64; no framework code)."""
from __future__ import annotations

import torch

F64 = torch.float64


def norm_rope(x, weight, eps, table, pos, rot, interleaved):
    """x [rows, heads, D] -> float64; table [P, rot]; pos [rows]."""
    x = x.to(F64)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.to(F64)
    out = y.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c, s = table[pos.long(), j].to(F64)[:, None], table[pos.long(), rot // 2 + j].to(F64)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def seen_slots(mode, window, sinks, ctx, n, i, p, mask_row=None):
    """Bool [ctx + n]: the slots that row i (at position p) of n rows sees."""
    out = torch.zeros(ctx + n, dtype=torch.bool)
    for s in range(ctx + n):
        near = window == 0 or s < sinks or s > p - window
        j = s - ctx
        if j < 0:
            out[s] = near
        elif mode == "causal":
            out[s] = j <= i and near
        elif mode == "full":
            out[s] = True
        else:
            out[s] = bool(mask_row[j])
    return out


def attention(q, k, v, scale, seen):
    """q [rows, hq, D], k / v [hkv, slots, D], seen [rows, slots] -> out, lse, the weighted |v| (for error bounds) and the
    largest sum of |q||k| of a seen pair times scale, all float64."""
    rows, hq, D = q.shape
    G = hq // k.shape[0]
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    out = torch.zeros(rows, hq, D, dtype=F64, device=q.device)
    absv = torch.zeros_like(out)
    lse = torch.full((rows, hq), float("-inf"), dtype=F64, device=q.device)
    big = 0.0
    for r in range(rows):
        at = seen[r].nonzero()[:, 0].to(q.device)
        if at.numel() == 0:
            continue
        for h in range(hq):
            kk, vv = k[h // G, at], v[h // G, at]
            s = (kk @ q[r, h]) * scale
            big = max(big, float(((kk.abs() @ q[r, h].abs()) * scale).max()))
            lse[r, h] = torch.logsumexp(s, 0)
            p = torch.softmax(s, 0)
            out[r, h], absv[r, h] = p @ vv, p @ vv.abs()
    return out, lse, absv, big


def sample(logits, gumbel, T, top_k, top_p, min_p):
    """One row: (token, logprob, margin): margin is how far the result is from another decision, over the draw, the
    boundary of top-p and that of min-p (only what could change the token counts)."""
    x = logits.to(F64)
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    top = float(x.max())
    if top == float("-inf"):
        return -1, float("-inf"), float("inf")
    if T == 0:
        return int((x == top).nonzero()[0, 0]), 0.0, float("inf")
    value, ids = torch.sort(x, descending=True, stable=True)
    if top_k > 0:
        value, ids = value[:top_k], ids[:top_k]
    w = torch.where(value == top, torch.ones_like(value), torch.exp((value - top) / T))
    before = torch.cumsum(w, 0) - w
    S = float(w.sum())
    kept = torch.ones_like(w, dtype=torch.bool) if top_p >= 1 else before < top_p * S
    kept &= w >= min_p
    score = value / T + gumbel.to(F64)[ids]
    sk = torch.where(kept, score, torch.full_like(score, float("-inf")))
    best = float(sk.max())
    token = int(ids[sk == best].min())
    at = int((ids == token).nonzero()[0, 0])
    rest = sk.clone()
    rest[at] = float("-inf")
    margin = best - float(rest.max()) if kept.sum() > 1 else float("inf")
    # Tokens near a boundary matter if they are the draw or would beat it.
    rival = (score >= best) if best > float("-inf") else torch.zeros_like(kept)
    if top_p < 1 and bool(rival.any()):
        margin = min(margin, float((before[rival] / S - top_p).abs().min()) + (0.0 if top_p * S < 1e30 else 0.0))
    if min_p > 0 and bool(rival.any()):
        margin = min(margin, float((w[rival] / min_p - 1).abs().min()))
    return token, float(torch.log(w[at] / w[kept].sum())), margin
