"""Two speculative cycles with the target's side on the library's kernels: a prompt enters one
attention layer's cache; a drafted chain, then a drafted tree, is verified by it.

    python examples/target_cycle.py

The target here is one attention layer between the embedding and the LM head (random weights;
projections are plain matrix products). What a real target's layers would do per cycle is what
it does: BlockAttention.append norms and rotates the block's queries and keys and puts its keys
and values into the cache, BlockAttention.attend lets the block see the past and itself (causal
for a chain, the ancestor mask for a tree), Sampler draws the target's tokens from the logits,
and the drafter's verification compares them with the draft. Rejected rows need no clean-up:
the cache's length says what is in it, and the next cycle writes over them.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from draft_head_gb300 import binding as B  # noqa: E402
from draft_head_gb300.runtime import DominoDrafter  # noqa: E402
from draft_head_gb300.target import BlockAttention, Sampler, rope_table  # noqa: E402


class Target:
    """Embedding, one attention layer with its cache, LM head."""

    def __init__(self, weights, drafter: DominoDrafter, batch: int, max_rows: int, capacity: int, n_q_heads=8, n_kv_heads=2,
                 head_dim=64, window=0, sinks=0, seed=1):
        self.w, self.dr, self.batch, self.hq, self.dim = weights, drafter, batch, n_q_heads, head_dim
        self.dev, d = weights["emb"].device, weights["emb"].shape[1]
        g = torch.Generator(device=self.dev)
        g.manual_seed(seed)
        rnd = lambda *s: (torch.randn(*s, generator=g, device=self.dev) * 0.05).to(torch.bfloat16)
        self.w_qkv, self.w_o = rnd((n_q_heads + 2 * n_kv_heads) * head_dim, d), rnd(d, n_q_heads * head_dim)
        self.k = torch.zeros(batch, n_kv_heads, capacity, head_dim, dtype=torch.bfloat16, device=self.dev)
        self.v = torch.zeros_like(self.k)
        ones = torch.ones(head_dim, dtype=torch.bfloat16, device=self.dev)
        self.attn = BlockAttention(self.k, self.v, n_q_heads, max_tokens=batch * max_rows, max_q=max_rows, max_ctx=capacity,
                                   window=window, sinks=sinks, rope=rope_table(capacity, head_dim, device=self.dev),
                                   q_weight=ones, k_weight=ones)
        self.ctx = torch.zeros(batch, dtype=torch.int32, device=self.dev)
        self.ws = B.workspace(256, self.dev)

    def hidden(self, tokens, q_start=None, positions=None, mask="causal"):
        """tokens [rows] of all requests, packed: the layer's output rows, bf16. They enter the cache at self.ctx."""
        x = torch.nn.functional.embedding(tokens.long(), self.w["emb"])
        q = self.attn.append(x @ self.w_qkv.T, self.ctx, q_start=q_start, positions=positions)
        out = self.attn.attend(q, self.ctx, q_start=q_start, positions=positions, mask=mask)
        return (x.float() * 20 + out.reshape(out.shape[0], -1) @ self.w_o.T).to(torch.bfloat16).contiguous()

    def logits(self, tokens, rows: int, **how):
        """A block of `rows` rows per request -> [batch * rows, V] fp32."""
        V = self.dr.head.V
        h = self.hidden(tokens, **how)
        out = torch.empty(self.batch * rows, V, dtype=torch.float32, device=self.dev)
        B.domino_base_logits(self.dr.head, h, self.batch, rows, out, None, self.ws)
        return out


def main(batch=3, P=7, n_nodes=8, top_m=16, V=2000, d=128, prompt=(40, 7, 23), seed=0, log=print):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda std, *s: (torch.randn(*s, generator=g, device=dev) * std).to(torch.bfloat16)
    gumbel = lambda rows: -torch.log(-torch.log(torch.rand(rows, V, generator=g, device=dev) * (1 - 2e-7) + 1e-7))
    G, r = 64, 32
    weights = dict(w_lm=rnd(d ** -0.5, V, d), emb=rnd(0.05, V, d), w_ih=rnd(0.05, 3 * G, d), w_hh=rnd(0.05, 3 * G, G), b_ih=rnd(0.02, 3 * G),
                   b_hh=rnd(0.02, 3 * G), w1=rnd(0.05, r, d + G), w2=rnd(0.05, V, r))
    dr = DominoDrafter(weights, batch, P, n_nodes=n_nodes, top_m=top_m)
    target = Target(weights, dr, batch, max(max(prompt), P + 1, n_nodes + 1), sum(prompt) + 4 * (P + n_nodes))
    settings = dict(temperature=torch.full((batch,), 0.8, device=dev), top_k=torch.full((batch,), 40, dtype=torch.int32, device=dev),
                    top_p=torch.full((batch,), 0.95, device=dev), min_p=torch.full((batch,), 0.02, device=dev))
    per_row = lambda rows: {k: v.repeat_interleave(rows).contiguous() for k, v in settings.items()}
    result = {"target": target, "drafter": dr, "gumbel": [], "logits": [], "tokens": [], "settings": settings}

    # The prompts, of unlike lengths, packed.
    start = torch.tensor([0] + list(prompt), device=dev).cumsum(0).to(torch.int32)
    prompts = torch.randint(0, V, (sum(prompt),), generator=g, device=dev, dtype=torch.int32)
    target.hidden(prompts, q_start=start)
    target.ctx += torch.tensor(prompt, dtype=torch.int32, device=dev)
    anchor = torch.randint(0, V, (batch,), generator=g, device=dev, dtype=torch.int32)

    # A chain: the anchor and P drafted tokens are P + 1 rows; row i's logits give the target's token i + 1.
    H = rnd(1.0, batch, P, d)
    drafted = dr.draft(H, anchor)
    block = torch.cat([anchor[:, None], drafted], 1)
    logits = target.logits(block.reshape(-1), P + 1)
    noise = gumbel(batch * (P + 1))
    sampler = Sampler(batch * (P + 1), V)
    drawn = sampler.sample(logits, noise, **per_row(P + 1)).view(batch, P + 1)
    result["logits"].append(logits)
    result["gumbel"].append(noise)
    result["tokens"].append(drawn.clone())
    accept, advanced = dr.verify(drawn[:, :P].contiguous())
    anchor = drawn.gather(1, accept.long()[:, None]).squeeze(1)  # the target's own token after the accepted ones
    target.ctx += advanced
    log("chain: accepted", accept.tolist(), "past", target.ctx.tolist())

    # A tree: node rows, each at its depth, seeing its ancestors.
    dr.base(rnd(1.0, batch, P, d))
    token, parent, depth, _ = dr.tree(anchor)
    rows = n_nodes + 1
    _, _, _, mask = dr.tree_verify(torch.zeros(batch, rows, dtype=torch.int32, device=dev), want_path=False, want_mask=True)
    positions = (target.ctx[:, None] + depth.clamp(min=0)).reshape(-1).contiguous()
    logits = target.logits(token.clamp(min=0).reshape(-1), rows, positions=positions, mask=mask)
    noise = gumbel(batch * rows)
    drawn = Sampler(batch * rows, V).sample(logits, noise, **per_row(rows))
    result["logits"].append(logits)
    result["gumbel"].append(noise)
    result["tokens"].append(drawn)
    accept, advanced, path, _ = dr.tree_verify(drawn.view(batch, rows), want_mask=False)
    # The accepted path's keys and values move to the slots of a chain (nodes lie in pop order).
    at = torch.arange(rows, device=dev)[None]
    keep = (path >= 0) & (at <= accept[:, None])
    src = (target.ctx[:, None] + torch.where(keep, path, at)).long()
    b = torch.arange(batch, device=dev)[:, None]
    for cache in (target.k, target.v):
        cache[b, :, (target.ctx[:, None] + at).long()] = cache[b, :, src]
    target.ctx += advanced
    log("tree: accepted", accept.tolist(), "past", target.ctx.tolist())
    status = [target.attn.last_status(), sampler.last_status(), dr.last_status()]
    log("device status", status)
    result.update(status=status, mask=mask, positions=positions, tree=(token, parent, depth))
    return result


if __name__ == "__main__":
    main()
