"""Cases of the operators around a paged key/value cache: new keys and values normed, rotated and
quantised as they are written to their pages, slots read back from their pages, attention of a
chunk of new tokens over the pages, and what the target's logits say of given tokens (their
log-probability and rank, the row's entropy and its most likely tokens). Sizes: the draft block of 16, the
tree of 16 nodes (17 rows with the root), the batches 1 / 16 / 64 and the vocabulary of this
repository's workloads; head counts, page sizes and context lengths are generic.

A quantised cache holds a head's vector of a slot as e4m3 codes and one power of two, its scale:
with 2^e the smallest power of two (of exponents -100 to 120) for which no element's magnitude is
above 448 * 2^e, the codes are x / 2^e rounded to nearest even, and the scale's byte is e + 127.
"""
import math
import random

import numpy as np
import torch

own = False

CAUSAL, FULL, TREE = "causal", "full", "tree"


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _append(name, cache, page, batch, rows, ctx, hq, hkv, dim, rot, pairs, norm, ragged):
    return {"name": name, "op": "append", "cache": cache, "page": page, "batch": batch, "rows": rows, "ctx": ctx, "hq": hq,
            "hkv": hkv, "dim": dim, "rot": rot, "pairs": pairs, "norm": norm, "ragged": ragged, "mix": 1}


def _read(name, cache, page, batch, ctx, hkv, dim, ragged):
    return {"name": name, "op": "read", "cache": cache, "page": page, "batch": batch, "rows": 0, "ctx": ctx, "hkv": hkv,
            "dim": dim, "ragged": ragged, "mix": 2}


def _attn(name, cache, page, batch, rows, ctx, hq, hkv, dim, mask, window, sinks, ragged):
    return {"name": name, "op": "attention", "cache": cache, "page": page, "batch": batch, "rows": rows, "ctx": ctx, "hq": hq,
            "hkv": hkv, "dim": dim, "mask": mask, "window": window, "sinks": sinks, "ragged": ragged, "mix": 3}


def _score(name, dtype, rows, vocab, top, peaked):
    return {"name": name, "op": "score", "dtype": dtype, "rows": rows, "vocab": vocab, "top": top, "peaked": peaked, "mix": 4}


def listed():
    return [
        # One request's draft block of 16 rows enters a quantised cache: the smallest call of a verification pass, latency.
        _append("append_block_b1", "e4m3", 64, 1, 16, 500, 32, 8, 128, 128, False, True, False),
        # A batch of prompts of unlike lengths entering a quantised cache: bandwidth.
        _append("append_prompts", "e4m3", 64, 4, 6000, 0, 32, 8, 128, 128, False, True, True),
        # Pages in bf16, an odd number of rows, no norm, half of each head rotated as neighbouring pairs.
        _append("append_bf16_pairs", "bf16", 16, 5, 173, 100, 14, 2, 64, 32, True, False, True),
        # One request's past leaves its pages, for a layer that wants it in one piece.
        _read("read_b1", "e4m3", 64, 1, 4000, 8, 128, False),
        # The pasts of 32 requests: bandwidth.
        _read("read_b32", "e4m3", 32, 32, 8000, 8, 128, True),
        # One request decoding one token over its quantised cache: latency.
        _attn("attn_token_b1", "e4m3", 64, 1, 1, 4000, 32, 8, 128, CAUSAL, 0, 0, False),
        # 128 requests decoding one token each over unlike pasts: bandwidth.
        _attn("attn_token_b128", "e4m3", 32, 128, 1, 8000, 32, 8, 128, CAUSAL, 0, 0, True),
        # 64 requests verify their draft blocks over pages in bf16, with a window and first tokens that stay visible: bandwidth.
        _attn("attn_block_b64", "bf16", 16, 64, 16, 8000, 32, 8, 128, CAUSAL, 4096, 4, True),
        # 16 requests verify their trees (root and 16 nodes, ancestor mask) over quantised pages.
        _attn("attn_tree_b16", "e4m3", 64, 16, 17, 6000, 32, 8, 128, TREE, 0, 0, True),
        # Prompts that enter in chunks: 4 requests with 2048 new tokens each over their pasts: the matrix products bound it.
        _attn("attn_chunks", "e4m3", 128, 4, 2048, 8000, 32, 8, 128, CAUSAL, 0, 0, True),
        # One row of the vocabulary, its 20 most likely tokens: latency.
        _score("score_b1", "f32", 1, 151936, 20, True),
        # The target's rows for 64 drafted trees: bandwidth.
        _score("score_trees_b64", "bf16", 1088, 151936, 8, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "score"])
    mix = rng.randrange(10, 1 << 20)
    cache = rng.choice(["e4m3", "e4m3", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128, 128])
    if op == "append":
        rows, batch = _log(rng, 1, 2000), _log(rng, 1, 64)
        while rows * batch > 16000:
            batch = max(1, batch // 2)
        return {"op": op, "cache": cache, "page": page, "batch": batch, "rows": rows, "ctx": _log(rng, 1, 500),
                "hq": hkv * rng.choice([1, 4, 5, 7]) if hkv < 8 else 32, "hkv": hkv, "dim": dim,
                "rot": rng.choice([0, dim, dim, dim // 2]), "pairs": rng.random() < 0.3, "norm": rng.random() < 0.7,
                "ragged": rng.random() < 0.7, "mix": mix}
    if op == "read":
        batch = _log(rng, 1, 32)
        return {"op": op, "cache": cache, "page": page, "batch": batch, "rows": 0, "ctx": _log(rng, 1, 8000), "hkv": hkv,
                "dim": dim, "ragged": rng.random() < 0.7, "mix": mix}
    if op == "attention":
        group = rng.choice([1, 4, 5, 8]) if hkv < 8 else 4
        form = rng.choice(["token", "block", "tree", "chunk"])
        ctx = _log(rng, 20, 12000)
        window = rng.choice([0, 0, _log(rng, 100, 4096)])
        rows, batch, mask = 1, _log(rng, 1, 64), CAUSAL
        if form == "block":
            rows, mask = rng.randrange(2, 24), rng.choice([CAUSAL, FULL])
        elif form == "tree":
            rows, mask = rng.randrange(2, 40), TREE
        elif form == "chunk":
            rows, batch, ctx = _log(rng, 50, 4000), rng.randrange(1, 4), _log(rng, 1, 6000)
        if cache == "f32":
            batch, ctx, rows = min(batch, 8), min(ctx, 3000), min(rows, 300)
        return {"op": op, "cache": cache, "page": page, "batch": batch, "rows": rows, "ctx": ctx, "hq": hkv * group, "hkv": hkv,
                "dim": dim, "mask": mask, "window": window, "sinks": rng.choice([0, 1, 4, 7]), "ragged": rng.random() < 0.7,
                "mix": mix}
    vocab = rng.choice([151936, 50257, 32000, _log(rng, 1000, 200000)])
    rows = max(1, min(_log(rng, 1, 1000), 150000000 // vocab))
    return {"op": op, "dtype": rng.choice(["bf16", "f32"]), "rows": rows, "vocab": vocab, "top": rng.choice([0, 1, 5, 8, 20, 32]),
            "peaked": rng.random() < 0.7, "mix": mix}


def _lengths(case):
    """Rows and past of each request: the case's own numbers, or with `ragged` unlike ones up to them."""
    rng = random.Random(case["mix"])
    b, n, c = case["batch"], case["rows"], case["ctx"]
    if not case["ragged"]:
        return [n] * b, [c] * b
    same_rows = n == 0 or case.get("mask") in (FULL, TREE)  # a draft block or a tree has the same rows for every request
    rows = [n if same_rows else max(1, round(n * rng.uniform(0.25, 1.0))) for _ in range(b)]
    ctx = [round(c * rng.uniform(0.05, 1.0)) for _ in range(b)]
    rows[0], ctx[-1] = n, c
    return rows, ctx


def _row_type(case):
    """The type of queries, keys and values as the layer computes them."""
    return torch.float32 if case["cache"] == "f32" else torch.bfloat16


def _generator(seed, case):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ---------------------------------------------------------------------------
# The quantised form: codes and the exponent's byte of vectors along the last axis.
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in 64 bits by its fields: a GPU's pow is a unit off for some."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x):
    part, power = torch.frexp(x.abs().amax(-1))  # part in [0.5, 1); 448 = 0.875 * 2^9
    e = (power - 9 + (part > 0.875)).clamp(-100, 120)
    codes = (x * _power(-e).to(x.dtype)[..., None]).float().to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scale):
    """What codes and scales stand for, in 32 bits (exact)."""
    return codes.float() * _power(scale.int() - 127).float()[..., None]


# ---------------------------------------------------------------------------
# What a program holds before the call.
# ---------------------------------------------------------------------------
def _prepare_pages(case, s, g):
    """Packed rows (q_start [batch + 1], ctx_len [batch], the host's bounds) and the pages: each request's are spread over a
    pool that holds a few more; table entries behind a request's last slot are -1."""
    rows, ctx = _lengths(case)
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    page, batch, hkv, dim = case["page"], case["batch"], case["hkv"], case["dim"]
    need = [(r + c + page - 1) // page for r, c in zip(rows, ctx)]
    total = sum(need) + 3
    s.update({"tokens": start[-1], "max_q": max(rows), "max_ctx": max(ctx), "max_pages": max(1, max(need)),
              "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
              "ctx_len": torch.tensor(ctx, dtype=torch.int32, device="cuda")})
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((batch, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
    need = torch.tensor(need, device="cuda")
    first = need.cumsum(0) - need
    at = torch.arange(s["max_pages"], device="cuda")[None, :]
    s["table"] = torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=total - 1)], table).contiguous()
    for kind in ("k", "v"):
        x = _normal(g, total, hkv, page, dim)
        if case["cache"] == "e4m3":
            s[kind + "_pages"], s[kind + "_scale"] = _quantise(x)
        else:
            s[kind + "_pages"], s[kind + "_scale"] = x.to(_row_type(case)), None


def _rope_table(positions, rot, base=1e6):
    """[positions, rot] fp32: the cosines of the rot / 2 angles, then their sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _tree(case, g):
    """The ancestor mask and depths of random trees [batch, rows]: node 0 the root, each other node below an earlier one."""
    b, n = case["batch"], case["rows"]
    u = torch.rand(b, n, generator=g, device="cuda")
    parent = (u * torch.arange(n, device="cuda")).long()
    seen = torch.eye(n, dtype=torch.bool, device="cuda").expand(b, n, n).clone()
    depth = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    at = torch.arange(b, device="cuda")
    for i in range(1, n):
        seen[:, i] |= seen[at, parent[:, i]]
        depth[:, i] = depth[at, parent[:, i]] + 1
    return seen.to(torch.uint8).contiguous(), depth


def prepare(case, seed):
    g = _generator(seed, case)
    s = {"case": dict(case)}
    if case["op"] == "score":
        rows, vocab, dt = case["rows"], case["vocab"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        logits = _normal(g, rows, vocab)
        if case["peaked"]:  # a model's rows: a broad bulk and a few likely tokens
            logits *= 2.0
            at = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")
            logits.scatter_add_(1, at, 14.0 * torch.rand(rows, 40, generator=g, device="cuda"))
        s["logits"] = logits.to(dt)
        # Given tokens: one of the likely ones in three rows of four, any one in the others, none in a few.
        likely = logits.argmax(1)
        anyone = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        u = torch.rand(rows, generator=g, device="cuda")
        tokens = torch.where(u < 0.75, likely, anyone)
        s["tokens"] = torch.where(u > 0.97, torch.full_like(tokens, -1), tokens).int()
        rng = random.Random(case["mix"] + 7)
        s["temperature"] = torch.tensor([rng.choice([0.6, 0.7, 0.8, 1.0]) for _ in range(rows)], device="cuda")
        if own:
            from draft_head_gb300.target import TokenScorer
            s["plan"] = TokenScorer(rows, vocab, dtype=dt, top_n=case["top"])
        return s
    _prepare_pages(case, s, g)
    hq, hkv, dim, dt = case.get("hq", case["hkv"]), case["hkv"], case["dim"], _row_type(case)
    if case["op"] == "append":
        s["qkv"] = (1.5 * _normal(g, s["tokens"], (hq + 2 * hkv) * dim)).to(dt)
        s["q_weight"] = (1.0 + 0.2 * _normal(g, dim)).to(dt)
        s["k_weight"] = (1.0 + 0.2 * _normal(g, dim)).to(dt)
        s["angles"] = _rope_table(s["max_ctx"] + s["max_q"], case["rot"]) if case["rot"] else None
        s["eps"] = 1e-6
    elif case["op"] == "read":
        s["k_out"] = torch.zeros(case["batch"], hkv, s["max_ctx"], dim, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        # Normed and rotated queries against normed keys: scores of spread about 2, as a trained layer has.
        s["q"] = (2.0 * _normal(g, s["tokens"], hq, dim)).to(dt)
        s["scale"] = dim ** -0.5
        s["mask"] = s["positions"] = None
        if case["mask"] == TREE:
            s["mask"], depth = _tree(case, g)
            s["positions"] = (s["ctx_len"][:, None] + depth).reshape(-1).to(torch.int32).contiguous()
    if own:
        from draft_head_gb300.target import PagedAttention
        normed = case.get("norm", True)
        s["plan"] = PagedAttention(s["k_pages"], s["v_pages"], s["table"], n_q_heads=hq, max_tokens=max(1, s["tokens"]),
                                   max_q=max(1, s["max_q"]), max_ctx=s["max_ctx"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   window=case.get("window", 0), sinks=case.get("sinks", 0), scale=s.get("scale"),
                                   rope=s.get("angles"), norm=normed, q_weight=s.get("q_weight") if normed else None,
                                   k_weight=s.get("k_weight") if normed else None, eps=s.get("eps", 1e-6),
                                   interleaved=case.get("pairs", False))
    return s


# ---------------------------------------------------------------------------
# One pass: the framework's calls, or the plain form.
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        p = s["plan"]
        if c["op"] == "append":
            q = p.append(s["qkv"], s["ctx_len"], q_start=s["q_start"])
            return _cache(s, q)
        if c["op"] == "read":
            p.read(s["k_out"], s["v_out"], s["ctx_len"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if c["op"] == "attention":
            out, lse = p.attend(s["q"], s["ctx_len"], q_start=s["q_start"], positions=s["positions"],
                                mask=s["mask"] if s["mask"] is not None else c["mask"], want_lse=True)
            return {"out": out, "lse": lse}
        r = p.score(s["logits"], s["tokens"], s["temperature"])
        return {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy, "top_ids": r.top_ids, "top_logprob": r.top_logprob}
    return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention, "score": _plain_score}[c["op"]](s)


def _cache(s, q):
    """What an append leaves: the queries and the pool, its codes and scales as the numbers that they are."""
    scales = {k: s[k].view(torch.float8_e8m0fnu) for k in ("k_scale", "v_scale") if s[k] is not None}
    return {"q": q, "k": s["k_pages"], "v": s["v_pages"], **scales}


def _request_of_rows(s):
    """For each packed row its request and its place in that request's rows."""
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    b = (t[:, None] >= s["q_start"][None, 1:]).sum(1)
    return b, t - s["q_start"][b]


def _plain_append(s):
    c = s["case"]
    hq, hkv, dim, rot, page = c["hq"], c["hkv"], c["dim"], c["rot"], c["page"]
    # What is quantised is computed in 64 bits: a value next to the border of two codes goes to the right one.
    x = s["qkv"].to(torch.float64 if c["cache"] == "e4m3" else torch.float32).view(s["tokens"], hq + 2 * hkv, dim)
    req, i = _request_of_rows(s)
    slot = (s["ctx_len"][req] + i).long()
    where = s["table"][req, slot // page].long()

    def turned(x, w):
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.to(x.dtype) if c["norm"] else x
        if not rot:
            return y
        row = s["angles"][slot][:, None, :].to(x.dtype)
        cos, sin = row[..., : rot // 2], row[..., rot // 2:]
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["pairs"] else (y[..., : rot // 2], y[..., rot // 2: rot])
        first, second = a * cos - b * sin, b * cos + a * sin
        z = torch.stack([first, second], -1).flatten(-2) if c["pairs"] else torch.cat([first, second], -1)
        return torch.cat([z, y[..., rot:]], -1)

    q = turned(x[:, :hq].float(), s["q_weight"]).to(s["qkv"].dtype)
    _put(s, "k", where, slot % page, turned(x[:, hq: hq + hkv], s["k_weight"]))
    _put(s, "v", where, slot % page, x[:, hq + hkv:])
    return _cache(s, q)


def _put(s, kind, where, at, x):
    if s[kind + "_scale"] is None:
        s[kind + "_pages"][where, :, at] = x.to(s[kind + "_pages"].dtype)
        return
    codes, scale = _quantise(x)
    s[kind + "_pages"].view(torch.uint8)[where, :, at] = codes.view(torch.uint8)
    s[kind + "_scale"][where, :, at] = scale


def _gathered(s, kind):
    """Every request's pages behind one another, [batch, hkv, max_pages * page, dim] in 32 bits."""
    c = s["case"]
    at = s["table"].clamp(min=0).long()
    pages = s[kind + "_pages"]
    if s[kind + "_scale"] is None:
        x = pages[at].float()
    else:
        x = _values(pages.view(torch.uint8)[at].view(torch.float8_e4m3fn), s[kind + "_scale"][at])
    return x.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["hkv"], -1, c["dim"])


def _plain_read(s):
    n = s["k_out"].shape[2]
    there = (torch.arange(n, device="cuda")[None, :] < s["ctx_len"][:, None])[:, None, :, None]
    for kind in ("k", "v"):
        s[kind + "_out"].copy_(torch.where(there, _gathered(s, kind)[:, :, :n].to(s["k_out"].dtype), s[kind + "_out"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _visible(s, req_rows, slots):
    """[batch, max_q, slots]: which slots each row sees, and which rows there are."""
    c = s["case"]
    i = torch.arange(s["max_q"], device="cuda")[None, :, None]
    slot = torch.arange(slots, device="cuda")[None, None, :]
    ctx = s["ctx_len"].long()[:, None, None]
    pos = ctx + i if s["positions"] is None else s["positions"].long()[req_rows][:, :, None]
    near = (slot < c["sinks"]) | (slot > pos - c["window"]) if c["window"] > 0 else torch.ones_like(slot, dtype=torch.bool)
    j = slot - ctx
    if c["mask"] == CAUSAL:
        block = (j <= i) & near
    elif c["mask"] == FULL:
        block = torch.ones_like(j, dtype=torch.bool)
    else:
        n = s["mask"].shape[-1]
        at = j.clamp(0, n - 1).expand(-1, n, -1)
        block = torch.gather(s["mask"].bool(), 2, at) & (j < n)
    rows = (s["q_start"][1:] - s["q_start"][:-1])[:, None, None]
    return torch.where(j < 0, near, block) & (j < rows) & (i < rows)


def _plain_attention(s):
    c = s["case"]
    b, hq, hkv, dim = c["batch"], c["hq"], c["hkv"], c["dim"]
    place = s["q_start"][:-1].long()[:, None] + torch.arange(s["max_q"], device="cuda")[None, :]
    place = place.clamp(max=s["tokens"] - 1)
    k = _gathered(s, "k")
    seen = _visible(s, place, k.shape[2])
    q = s["q"].float()[place].view(b, s["max_q"], hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(b, hkv, hq // hkv * s["max_q"], dim)
    score = (q @ k.transpose(-1, -2)).view(b, hkv, hq // hkv, s["max_q"], -1).mul_(s["scale"])
    del k
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = p.view(b, hkv, hq // hkv * s["max_q"], -1) @ _gathered(s, "v")
    out = out.view(b, hkv, hq // hkv, s["max_q"], dim) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    req, i = _request_of_rows(s)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, s["max_q"], hq, dim)[req, i]
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(b, s["max_q"], hq)[req, i]}


def _plain_score(s):
    z = s["logits"].float() / s["temperature"][:, None]
    top = z.amax(1, keepdim=True)
    d = z - top
    w = d.exp()
    total = w.sum(1)
    lse = total.log()  # from the maximum
    entropy = lse - (w * d).sum(1) / total
    token = s["tokens"].long()
    at = token.clamp(min=0)[:, None]
    logprob = torch.gather(d, 1, at).squeeze(1) - lse
    raw = s["logits"].float()
    mine = torch.gather(raw, 1, at)
    ids = torch.arange(raw.shape[1], device="cuda")[None, :]
    rank = ((raw > mine) | ((raw == mine) & (ids < at))).sum(1)
    value, order = torch.sort(raw, dim=1, descending=True, stable=True)  # ties go to the lowest token id
    order = order[:, : s["case"]["top"]]
    none = token < 0
    return {"logprob": torch.where(none, torch.zeros_like(logprob), logprob),
            "rank": torch.where(none, torch.zeros_like(rank), rank).int(), "entropy": entropy, "top_ids": order.int(),
            "top_logprob": torch.gather(d, 1, order) - lse[:, None]}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def _pairs(case):
    """Row-slot pairs that are seen, and slots that any row of their request sees, over all requests (one head). Trees, whose
    depths differ from seed to seed, are counted at four ancestors a node."""
    pairs = slots = 0
    for n, c in zip(*_lengths(case)):
        w, k = case["window"], case["sinks"]
        i = np.arange(n, dtype=np.int64)
        pos = c + i if case["mask"] != TREE else c + np.minimum(i, 4)
        low = np.maximum(0, pos - w + 1) if w > 0 else np.zeros_like(pos)
        first = np.minimum(low, c)
        past = c - first + np.minimum(k, first)
        if case["mask"] == CAUSAL:
            lo = np.maximum(low, c)
            block = pos + 1 - lo + np.clip(np.minimum(k, lo) - c, 0, None)
        elif case["mask"] == FULL:
            block = np.full(n, n)
        else:
            block = np.minimum(i, 4) + 1
        pairs += int((past + block).sum())
        slots += n + int(past.max())
    return pairs, slots


def work(case):
    if case["op"] == "score":
        rows, vocab, size = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * (vocab * size + 4 + 4 + 12 + 8 * case["top"]), "flops": 5 * rows * vocab}
    rows, ctx = _lengths(case)
    tokens, hkv, dim = sum(rows), case["hkv"], case["dim"]
    size = 4 if case["cache"] == "f32" else 2  # of queries, keys and values outside the pages
    vector = dim + 1 if case["cache"] == "e4m3" else dim * size  # of a head's vector in a page
    if case["op"] == "append":
        values = tokens * (case["hq"] + 2 * hkv) * dim
        return {"bytes": values * size + tokens * case["hq"] * dim * size + 2 * tokens * hkv * vector + tokens * case["rot"] * 4,
                "flops": 7 * values}
    if case["op"] == "read":
        return {"bytes": 2 * sum(ctx) * hkv * (vector + dim * size), "flops": 2 * sum(ctx) * hkv * dim}
    pairs, slots = _pairs(case)
    hq = case["hq"]
    return {"bytes": 2 * tokens * hq * dim * size + 2 * slots * hkv * vector + 4 * tokens * hq, "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention, "score": _exact_score}[case["op"]](case, s)


def _exact_slots(s, kind, b, n):
    """The first n slots of request b, [hkv, n, dim] in 64 bits."""
    page = s["case"]["page"]
    ids = s["table"][b, : max(1, (n + page - 1) // page)].clamp(min=0).tolist()
    pages = [s[kind + "_pages"][i].double() for i in ids]
    if s[kind + "_scale"] is not None:
        pages = [x * _power(s[kind + "_scale"][i].int() - 127)[..., None] for x, i in zip(pages, ids)]
    return torch.cat(pages, 1)[:, :n]


def _nearest_codes(x):
    """Vectors [..., dim] in 64 bits as (the numbers of their codes, their scales): a search through the 127 magnitudes."""
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    e = torch.full(x.shape[:-1], -100, device=x.device)
    most = x.abs().amax(-1)
    while bool((most > 448 * _power(e)).any()):
        e = torch.where(most > 448 * _power(e), e + 1, e)
    y = x / _power(e)[..., None]
    between = (grid[1:] + grid[:-1]) / 2
    at = torch.bucketize(y.abs(), between)  # a tie goes below it,
    tie = (y.abs() == between[at.clamp(max=125)]) & (at < 126) & (at % 2 == 1)
    return torch.copysign(grid[at + tie], y), _power(e)  # or to the even code


def _exact_append(c, s):
    hq, hkv, dim, rot, page = c["hq"], c["hkv"], c["dim"], c["rot"], c["page"]
    heads = s["qkv"].double().view(s["tokens"], hq + 2 * hkv, dim)
    pools = {k: s[k + "_pages"].double() for k in "kv"}
    scales = {k: None if s[k + "_scale"] is None else _power(s[k + "_scale"].int() - 127) for k in "kv"}
    first = torch.arange(0, rot, 2, device="cuda") if c["pairs"] else torch.arange(rot // 2, device="cuda")
    second = first + 1 if c["pairs"] else first + rot // 2
    out = torch.empty(s["tokens"], hq, dim, dtype=torch.float64, device="cuda")
    begin = 0
    for b, (n, ctx) in enumerate(zip(*_lengths(c))):
        x = heads[begin: begin + n].clone()
        if c["norm"]:
            w = torch.ones(hq + 2 * hkv, dim, dtype=torch.float64, device="cuda")
            w[:hq], w[hq: hq + hkv] = s["q_weight"].double(), s["k_weight"].double()
            x[:, : hq + hkv] /= (x[:, : hq + hkv].square().sum(-1, keepdim=True) / dim + s["eps"]).sqrt()
            x *= w
        if rot:
            angle = s["angles"][ctx: ctx + n].double()
            e = torch.complex(angle[:, : rot // 2], angle[:, rot // 2:])[:, None]
            y = x[:, : hq + hkv]
            z = torch.complex(y[..., first], y[..., second]) * e
            y[..., first], y[..., second] = z.real, z.imag
        out[begin: begin + n] = x[:, :hq]
        slot = torch.arange(ctx, ctx + n, device="cuda")
        where, at = s["table"][b].long()[slot // page], slot % page
        for kind, part in (("k", x[:, hq: hq + hkv]), ("v", x[:, hq + hkv:])):
            if scales[kind] is None:
                pools[kind][where, :, at] = part
            else:
                pools[kind][where, :, at], scales[kind][where, :, at] = _nearest_codes(part)
        begin += n
    kept = {k + "_scale": v for k, v in scales.items() if v is not None}
    return {"q": out, "k": pools["k"], "v": pools["v"], **kept}


def _exact_read(c, s):
    outs = {}
    for kind in "kv":
        o = s[kind + "_out"].double()
        for b, n in enumerate(_lengths(c)[1]):
            o[b, :, :n] = _exact_slots(s, kind, b, n)
        outs[kind] = o
    return outs


def _exact_attention(c, s):
    hq, hkv, dim = c["hq"], c["hkv"], c["dim"]
    out = torch.zeros(s["tokens"], hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    begin = 0
    for b, (n, ctx) in enumerate(zip(*_lengths(c))):
        k, v = _exact_slots(s, "k", b, ctx + n), _exact_slots(s, "v", b, ctx + n)
        for r0 in range(0, n, 2048):  # rows in pieces, so that the scores fit
            r1 = min(n, r0 + 2048)
            rows = torch.arange(r0, r1, device="cuda")
            keys = torch.arange(ctx + n, device="cuda")
            pos = ctx + rows if s["positions"] is None else s["positions"][begin + r0: begin + r1].long()
            allowed = torch.ones(r1 - r0, ctx + n, dtype=torch.bool, device="cuda")
            if c["window"]:
                allowed = (keys[None] < c["sinks"]) | (pos[:, None] - keys[None] < c["window"])
            if c["mask"] == CAUSAL:
                allowed &= keys[None] <= ctx + rows[:, None]
            elif c["mask"] == FULL:
                allowed[:, ctx:] = True
            else:
                allowed[:, ctx:] = s["mask"][b, r0:r1, :n] != 0
            for h in range(hq):
                score = s["q"][begin + r0: begin + r1, h].double() @ k[h * hkv // hq].T
                score = torch.where(allowed, score * s["scale"], -math.inf)
                lse[begin + r0: begin + r1, h] = torch.logsumexp(score, 1)
                p = torch.softmax(score, 1).nan_to_num(0.0)
                out[begin + r0: begin + r1, h] = p @ v[h * hkv // hq]
        begin += n
    return {"out": out, "lse": lse}


def _exact_score(c, s):
    rows, n = c["rows"], c["top"]
    logprob, rank, entropy, top = [], [], [], []
    ids = torch.empty(rows, n, dtype=torch.int32)
    t, given = s["temperature"].tolist(), s["tokens"].tolist()
    for r in range(rows):
        raw = s["logits"][r].double()
        lp = torch.log_softmax(raw / t[r], 0)
        entropy.append(float(-(lp.exp() * lp).sum()))
        value, order = raw.sort(descending=True, stable=True)
        logprob.append(float(lp[given[r]]) if given[r] >= 0 else 0.0)
        rank.append(int((order == given[r]).nonzero()[0, 0]) if given[r] >= 0 else 0)
        ids[r] = order[:n].int().cpu()
        top.append(lp[order[:n]].cpu())
    f64 = lambda x: torch.tensor(x, dtype=torch.float64)  # noqa: E731
    return {"logprob": f64(logprob), "rank": torch.tensor(rank, dtype=torch.int32), "entropy": f64(entropy), "top_ids": ids,
            "top_logprob": torch.stack(top)}
