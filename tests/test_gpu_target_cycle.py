"""The example that runs the target-side operators together with the drafter:
its draws are the 64-bit draws from its own logits, its statuses are clean, and
the tree's logits are those of each node's root path run as a plain causal block
(the ancestor mask, the positions and the cache agree)."""
import os
import sys

import pytest
import torch

from tests import target_oracle as O

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_target_cycle_example():
    import target_cycle as T
    lines = []
    r = T.main(log=lambda *a: lines.append(a))
    torch.cuda.synchronize()
    assert r["status"] == [0, 0, 0] and len(lines) == 3
    batch = 3
    for logits, noise, tokens in zip(r["logits"], r["gumbel"], r["tokens"]):
        assert bool(torch.isfinite(logits).all())
        tokens, compared = tokens.reshape(-1).tolist(), 0
        for x in range(logits.shape[0]):
            want, _, margin = O.sample(logits[x], noise[x], 0.8, 40, 0.95, 0.02)
            if margin > 1e-4:
                compared += 1
                assert tokens[x] == want
        assert compared > logits.shape[0] // 2

    # Each node's path from the root, as a causal block over the same past: same logits at its end.
    target, (token, parent, depth) = r["target"], r["tree"]
    rows = token.shape[1]
    past = target.ctx - r["drafter"].advanced
    tree_logits = r["logits"][1].view(batch, rows, -1)
    k0, v0, ctx0 = target.k.clone(), target.v.clone(), target.ctx.clone()
    target.ctx = past
    for node in range(rows):
        paths = []
        for b in range(batch):
            p, n = [], node
            while n >= 0:
                p.append(int(token[b, n]))
                n = int(parent[b, n])
            paths.append(p[::-1])
        lens = [len(p) for p in paths]
        start = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        flat = torch.tensor(sum(paths, []), dtype=torch.int32, device="cuda")
        h = target.hidden(flat, q_start=start)
        last = h[(start[1:] - 1).long()].float() @ target.w["w_lm"].float().T
        for b in range(batch):
            assert lens[b] == int(depth[b, node]) + 1
            # bf16 rows: two roundings of the layer's output apart, 2^-7 of a logit's terms
            bound = 2.0 ** -7 * float((h[start[b + 1] - 1].float().abs() @ target.w["w_lm"].float().abs().T).max())
            assert float((last[b] - tree_logits[b, node]).abs().max()) <= bound
        target.k.copy_(k0)
        target.v.copy_(v0)
    target.ctx = ctx0
