"""Cases of the operators around the target's pass over a drafted block: the per-head
norm and rotation that fills the key/value cache, attention of the block's rows over
that cache, and the draw from the target's logits. Sizes: the draft block of 16, the
tree of 16 nodes (17 rows with the root), the batches 1 / 16 / 64 and the vocabulary of
this repository's workloads; head counts and context lengths are generic.
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
def _rope(name, dtype, batch, rows, ctx, hq, hkv, dim, rot, pairs, ragged):
    return {"name": name, "op": "rope", "dtype": dtype, "batch": batch, "rows": rows, "ctx": ctx, "hq": hq, "hkv": hkv,
            "dim": dim, "rot": rot, "pairs": pairs, "ragged": ragged, "mix": 1}


def _attn(name, dtype, batch, rows, ctx, hq, hkv, dim, mask, window, sinks, ragged):
    return {"name": name, "op": "attention", "dtype": dtype, "batch": batch, "rows": rows, "ctx": ctx, "hq": hq,
            "hkv": hkv, "dim": dim, "mask": mask, "window": window, "sinks": sinks, "ragged": ragged, "mix": 2}


def _sample(name, dtype, rows, vocab, kind, peaked):
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "kind": kind, "peaked": peaked,
            "mix": 3}


def listed():
    return [
        # One request's draft block of 16 rows: the smallest call of a verification pass, latency.
        _rope("rope_block_b1", "bf16", 1, 16, 48, 32, 8, 128, 128, False, False),
        # A batch of prompts of unlike lengths entering the cache: bandwidth.
        _rope("rope_prompts", "bf16", 4, 6000, 0, 32, 8, 128, 128, False, True),
        # fp32 heads of an odd number of rows, half of each head rotated, neighbouring pairs.
        _rope("rope_f32_pairs", "f32", 5, 173, 100, 14, 2, 64, 32, True, True),
        # One request decoding one token over its whole cache: latency.
        _attn("attn_token_b1", "bf16", 1, 1, 4000, 32, 8, 128, CAUSAL, 0, 0, False),
        # 64 requests, the draft block's rows see each other both ways; window and sinks over unlike contexts: bandwidth.
        _attn("attn_block_b64", "bf16", 64, 16, 8000, 32, 8, 128, FULL, 4096, 4, True),
        # 16 requests verify their trees (root and 16 nodes, ancestor mask) over unlike contexts.
        _attn("attn_tree_b16", "bf16", 16, 17, 6000, 32, 8, 128, TREE, 0, 0, True),
        # Two prompts, causal with window and sinks: the matrix products bound it.
        _attn("attn_prompts_window", "bf16", 2, 8192, 0, 32, 8, 128, CAUSAL, 2048, 4, True),
        # fp32, a head size that is no power of two, a few rows each.
        _attn("attn_f32_ragged", "f32", 3, 40, 1500, 6, 2, 80, CAUSAL, 700, 3, True),
        # One row of the vocabulary with all filters: latency.
        _sample("sample_b1", "f32", 1, 151936, "all", True),
        # The target's rows for 64 draft blocks, each request with its own settings: bandwidth.
        _sample("sample_blocks_b64", "f32", 1024, 151936, "mixed", True),
        # 16 trees at top-p alone over flat rows (logits of spread 1, this repository's synthetic ones): most of the
        # vocabulary stays in.
        _sample("sample_trees_flat", "f32", 272, 151936, "top_p", False),
        # bf16 logits, an odd vocabulary whose rows are not aligned.
        _sample("sample_bf16_odd", "bf16", 37, 50257, "mixed", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "sample"])
    mix = rng.randrange(1, 1 << 20)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 128])
        rows, batch = _log(rng, 1, 2000), _log(rng, 1, 64)
        while rows * batch > 16000:
            batch = max(1, batch // 2)
        return {"op": op, "dtype": dtype, "batch": batch, "rows": rows, "ctx": _log(rng, 1, 500), "hq": hkv * rng.choice([1, 4, 5, 7]) if hkv < 8 else 32,
                "hkv": hkv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2]), "pairs": rng.random() < 0.3,
                "ragged": rng.random() < 0.7, "mix": mix}
    if op == "attention":
        hkv = rng.choice([2, 4, 8])
        group = rng.choice([1, 4, 5, 8]) if hkv < 8 else 4
        form = rng.choice(["token", "block", "tree", "prompt"])
        ctx = _log(rng, 20, 12000)
        window = rng.choice([0, 0, _log(rng, 100, 4096)])
        rows, batch, mask = 1, _log(rng, 1, 64), CAUSAL
        if form == "block":
            rows, mask = rng.randrange(2, 24), rng.choice([CAUSAL, FULL])
        elif form == "tree":
            rows, mask = rng.randrange(2, 40), TREE
        elif form == "prompt":
            rows, batch, ctx = _log(rng, 50, 5000), rng.randrange(1, 3), _log(rng, 1, 3000)
        if dtype == "f32":
            batch, ctx, rows = min(batch, 8), min(ctx, 3000), min(rows, 300)
        return {"op": op, "dtype": dtype, "batch": batch, "rows": rows, "ctx": ctx, "hq": hkv * group, "hkv": hkv,
                "dim": rng.choice([64, 128, 128, 80]) if form != "prompt" else rng.choice([64, 128]), "mask": mask, "window": window,
                "sinks": rng.choice([0, 1, 4, 7]), "ragged": rng.random() < 0.7, "mix": mix}
    vocab = rng.choice([151936, 50257, 32000, _log(rng, 1000, 200000)])
    rows = max(1, min(_log(rng, 1, 1000), 150000000 // vocab))
    return {"op": op, "dtype": dtype, "rows": rows, "vocab": vocab, "kind": rng.choice(["all", "mixed", "mixed", "top_p", "top_k", "min_p", "plain"]),
            "peaked": rng.random() < 0.7, "mix": mix}


def _lengths(case):
    """Rows and context of each request: the case's own numbers, or with `ragged` unlike ones up to them."""
    rng = random.Random(case["mix"])
    b, n, c = case["batch"], case["rows"], case["ctx"]
    if not case["ragged"]:
        return [n] * b, [c] * b
    same_rows = case.get("mask") in (FULL, TREE)  # a draft block or a tree has the same rows for every request
    rows = [n if same_rows else max(1, round(n * rng.uniform(0.25, 1.0))) for _ in range(b)]
    ctx = [round(c * rng.uniform(0.05, 1.0)) for _ in range(b)]
    rows[0], ctx[-1] = n, c
    return rows, ctx


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _generator(seed, case):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ---------------------------------------------------------------------------
# What a program holds before the call.
# ---------------------------------------------------------------------------
def _prepare_rows(case):
    """Packed rows: q_start [batch + 1], ctx_len [batch], and the host's bounds."""
    rows, ctx = _lengths(case)
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    return {"tokens": start[-1], "max_q": max(rows), "max_ctx": max(ctx), "capacity": max(r + c for r, c in zip(rows, ctx)),
            "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
            "ctx_len": torch.tensor(ctx, dtype=torch.int32, device="cuda")}


def _rope_table(positions, rot, base=1e6):
    """[positions, rot] fp32: the cosines of the rot / 2 angles, then their sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _tree(case, g):
    """Parents, depths and the ancestor mask of random trees [batch, rows]: node 0 the root, each other node below an earlier one."""
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
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        logits = _normal(g, rows, vocab)
        if case["peaked"]:  # a model's rows: a broad bulk and a few likely tokens
            logits *= 2.0
            at = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")
            logits.scatter_add_(1, at, 14.0 * torch.rand(rows, 40, generator=g, device="cuda"))
        s["logits"] = logits.to(_dtype(case))
        u = (torch.randint(0, 1 << 24, (rows, vocab), generator=g, device="cuda").float() + 0.5) / float(1 << 24)
        s["gumbel"] = u.log_().neg_().log_().neg_()
        rng = random.Random(case["mix"] + 7)
        kind = case["kind"]
        pick = lambda k, some: [rng.choice(some) if kind in (k, "all", "mixed") else None for _ in range(rows)]
        off = lambda v, none: [none if (x is None or (kind == "mixed" and rng.random() < 0.4)) else x for x in v]
        t = [rng.choice([0.6, 0.7, 0.8, 1.0]) for _ in range(rows)]
        if kind == "mixed":
            t = [0.0 if rng.random() < 0.1 else x for x in t]
        s["temperature"] = torch.tensor(t, device="cuda")
        s["top_k"] = torch.tensor(off(pick("top_k", [20, 40, 64, 1000]), 0), dtype=torch.int32, device="cuda")
        s["top_p"] = torch.tensor(off(pick("top_p", [0.8, 0.9, 0.95]), 1.0), device="cuda")
        s["min_p"] = torch.tensor(off(pick("min_p", [0.02, 0.05, 0.1]), 0.0), device="cuda")
        if own:
            from draft_head_gb300.target import Sampler
            s["plan"] = Sampler(rows, vocab, dtype=_dtype(case))
        return s
    s.update(_prepare_rows(case))
    b, hq, hkv, dim, dt = case["batch"], case["hq"], case["hkv"], case["dim"], _dtype(case)
    s["k_cache"] = _normal(g, b, hkv, s["capacity"], dim).to(dt)
    s["v_cache"] = _normal(g, b, hkv, s["capacity"], dim).to(dt)
    if case["op"] == "rope":
        s["qkv"] = (1.5 * _normal(g, s["tokens"], (hq + 2 * hkv) * dim)).to(dt)
        s["q_weight"] = (1.0 + 0.2 * _normal(g, dim)).to(dt)
        s["k_weight"] = (1.0 + 0.2 * _normal(g, dim)).to(dt)
        s["table"] = _rope_table(s["capacity"], case["rot"])
        s["eps"] = 1e-6
    else:
        # Normed and rotated queries against normed keys: scores of spread about 2, as a trained layer has.
        s["q"] = (2.0 * _normal(g, s["tokens"], hq, dim)).to(dt)
        s["scale"] = dim ** -0.5
        s["mask"] = s["positions"] = None
        if case["mask"] == TREE:
            s["mask"], depth = _tree(case, g)
            s["positions"] = (s["ctx_len"][:, None] + depth).reshape(-1).to(torch.int32).contiguous()
    if own:
        from draft_head_gb300.target import BlockAttention
        s["plan"] = BlockAttention(s["k_cache"], s["v_cache"], n_q_heads=hq, max_tokens=s["tokens"], max_q=s["max_q"],
                                   max_ctx=s["max_ctx"], window=case.get("window", 0), sinks=case.get("sinks", 0),
                                   scale=s.get("scale"), rope=s.get("table"), q_weight=s.get("q_weight"),
                                   k_weight=s.get("k_weight"), eps=s.get("eps", 1e-6), interleaved=case.get("pairs", False))
    return s


# ---------------------------------------------------------------------------
# One pass: the framework's calls, or the plain form.
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        p = s["plan"]
        if op == "rope":
            q = p.append(s["qkv"], s["ctx_len"], q_start=s["q_start"])
            return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
        if op == "attention":
            out, lse = p.attend(s["q"], s["ctx_len"], q_start=s["q_start"], positions=s["positions"],
                                mask=s["mask"] if s["mask"] is not None else s["case"]["mask"], want_lse=True)
            return {"out": out, "lse": lse}
        tokens, logprob = p.sample(s["logits"], s["gumbel"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], want_logprob=True)
        return {"tokens": tokens, "logprob": logprob}
    return {"rope": _plain_rope, "attention": _plain_attention, "sample": _plain_sample}[op](s)


def _request_of_rows(s):
    """For each packed row its request and its place in that request's block."""
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    b = (t[:, None] >= s["q_start"][None, 1:]).sum(1)
    return b, t - s["q_start"][b]


def _plain_rope(s):
    c = s["case"]
    hq, hkv, dim, rot = c["hq"], c["hkv"], c["dim"], c["rot"]
    x = s["qkv"].float().view(s["tokens"], hq + 2 * hkv, dim)
    req, i = _request_of_rows(s)
    slot = s["ctx_len"][req] + i
    row = s["table"][slot][:, None, :]
    cos, sin = row[..., : rot // 2], row[..., rot // 2:]

    def turned(x, w):
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["pairs"] else (y[..., : rot // 2], y[..., rot // 2: rot])
        first, second = a * cos - b * sin, b * cos + a * sin
        z = torch.stack([first, second], -1).flatten(-2) if c["pairs"] else torch.cat([first, second], -1)
        return torch.cat([z, y[..., rot:]], -1)

    dt = s["qkv"].dtype
    q = turned(x[:, :hq], s["q_weight"]).to(dt)
    s["k_cache"][req, :, slot] = turned(x[:, hq: hq + hkv], s["k_weight"]).to(dt)
    s["v_cache"][req, :, slot] = x[:, hq + hkv:].to(dt)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _visible(s, req_rows):
    """[batch, max_q, capacity]: which slots each row sees, and which rows there are."""
    c = s["case"]
    i = torch.arange(s["max_q"], device="cuda")[None, :, None]
    slot = torch.arange(s["capacity"], device="cuda")[None, None, :]
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
    seen = _visible(s, place)
    q = s["q"].float()[place].view(b, s["max_q"], hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(b, hkv, hq // hkv * s["max_q"], dim)
    score = (q @ s["k_cache"].float().transpose(-1, -2)).view(b, hkv, hq // hkv, s["max_q"], -1).mul_(s["scale"])
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = p.view(b, hkv, hq // hkv * s["max_q"], -1) @ s["v_cache"].float()
    out = out.view(b, hkv, hq // hkv, s["max_q"], dim) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    req, i = _request_of_rows(s)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, s["max_q"], hq, dim)[req, i]
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(b, s["max_q"], hq)[req, i]}


def _plain_sample(s):
    logits = s["logits"].float()
    order_value, order = torch.sort(logits, dim=1, descending=True, stable=True)
    t = s["temperature"][:, None]
    greedy = t == 0
    z = order_value / torch.where(greedy, torch.ones_like(t), t)
    w = (z - z[:, :1]).exp()
    rank = torch.arange(z.shape[1], device="cuda")[None, :]
    k = s["top_k"][:, None]
    keep = (k == 0) | (rank < k)
    w = torch.where(keep, w, torch.zeros_like(w))
    mass = w.cumsum(1)
    keep &= ((mass - w) < s["top_p"][:, None] * w.sum(1, keepdim=True)) | (s["top_p"][:, None] >= 1)
    keep &= w >= s["min_p"][:, None]
    keep = torch.where(greedy, rank == 0, keep)
    total = torch.where(keep, w, torch.zeros_like(w)).sum(1)
    score = torch.where(keep, z + torch.gather(s["gumbel"], 1, order), torch.full_like(z, float("-inf")))
    best = score.amax(1, keepdim=True)
    # ties go to the lowest token id
    token = torch.where((score == best) & keep, order, torch.full_like(order, z.shape[1])).amin(1)
    at = (order == token[:, None]).to(torch.uint8).argmax(1, keepdim=True)
    logprob = torch.gather(z - z[:, :1], 1, at).squeeze(1) - total.log()
    return {"tokens": token.to(torch.int32), "logprob": torch.where(greedy[:, 0], torch.zeros_like(logprob), logprob)}


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
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        return {"bytes": rows * (vocab * size + 8 + 16 + 4), "flops": 4 * rows * vocab}
    tokens = sum(_lengths(case)[0])
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "rope":
        values = tokens * (hq + 2 * hkv) * dim
        return {"bytes": 2 * values * size + tokens * case["rot"] * 4, "flops": 7 * values}
    pairs, slots = _pairs(case)
    return {"bytes": 2 * tokens * hq * dim * size + 2 * slots * hkv * dim * size + 4 * tokens * hq, "flops": 4 * pairs * hq * dim}


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
    return {"rope": _exact_rope, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](case, s)


def _exact_rope(c, s):
    hq, hkv, dim, rot = c["hq"], c["hkv"], c["dim"], c["rot"]
    heads = s["qkv"].double().view(s["tokens"], hq + 2 * hkv, dim)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    first = torch.arange(0, rot, 2, device="cuda") if c["pairs"] else torch.arange(rot // 2, device="cuda")
    second = first + 1 if c["pairs"] else first + rot // 2
    out = torch.empty(s["tokens"], hq, dim, dtype=torch.float64, device="cuda")
    begin = 0
    for b, (n, ctx) in enumerate(zip(*_lengths(c))):
        x = heads[begin: begin + n]
        angle = s["table"][ctx: ctx + n].double()
        e = torch.complex(angle[:, : rot // 2], angle[:, rot // 2:])[:, None]
        for part, weight, to in ((x[:, :hq], s["q_weight"], None), (x[:, hq: hq + hkv], s["k_weight"], k_cache)):
            y = part / (part.square().sum(-1, keepdim=True) / dim + s["eps"]).sqrt() * weight.double()
            turned = torch.complex(y[..., first], y[..., second]) * e
            y[..., first], y[..., second] = turned.real, turned.imag
            if to is None:
                out[begin: begin + n] = y
            else:
                to[b, :, ctx: ctx + n] = y.transpose(0, 1)
        v_cache[b, :, ctx: ctx + n] = x[:, hq + hkv:].transpose(0, 1)
        begin += n
    return {"q": out, "k": k_cache, "v": v_cache}


def _exact_attention(c, s):
    hq, hkv, dim = c["hq"], c["hkv"], c["dim"]
    out = torch.zeros(s["tokens"], hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    begin = 0
    for b, (n, ctx) in enumerate(zip(*_lengths(c))):
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
                score = s["q"][begin + r0: begin + r1, h].double() @ s["k_cache"][b, h * hkv // hq, : ctx + n].double().T
                score = torch.where(allowed, score * s["scale"], -math.inf)
                lse[begin + r0: begin + r1, h] = torch.logsumexp(score, 1)
                p = torch.softmax(score, 1).nan_to_num(0.0)
                out[begin + r0: begin + r1, h] = p @ s["v_cache"][b, h * hkv // hq, : ctx + n].double()
        begin += n
    return {"out": out, "lse": lse}


def _exact_sample(c, s):
    tokens, logprob = [], []
    k, p, m, t = (s[x].tolist() for x in ("top_k", "top_p", "min_p", "temperature"))
    for r in range(c["rows"]):
        raw = s["logits"][r].double()
        if t[r] == 0:
            tokens.append(int((raw == raw.max()).nonzero()[0, 0]))
            logprob.append(0.0)
            continue
        value, ids = raw.sort(descending=True, stable=True)
        if k[r]:
            value, ids = value[: k[r]], ids[: k[r]]
        prob = torch.softmax(value / t[r], 0)
        before = prob.cumsum(0) - prob
        kept = (before < p[r]) if p[r] < 1 else torch.ones_like(prob, dtype=torch.bool)
        kept &= prob >= m[r] * prob[0]
        prob, ids, value = prob[kept], ids[kept], value[kept]
        best = int((value / t[r] + s["gumbel"][r].double()[ids]).argmax())
        tokens.append(int(ids[best]))
        logprob.append(float((prob[best] / prob.sum()).log()))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "logprob": torch.tensor(logprob, dtype=torch.float64)}
