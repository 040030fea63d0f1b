"""The example over a cache in pages: append, attend, score and the moves of a tree's slots together, with the drafter."""
import os
import sys

import pytest
import torch

from tests import paged_oracle as P
from tests import target_oracle as O

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

KINDS = [torch.bfloat16, torch.float8_e4m3fn]


@pytest.mark.parametrize("kind", KINDS)
def test_target_cycle_over_pages(kind):
    import target_cycle as T
    lines = []
    r = T.main(log=lambda *a: lines.append(a), pages=kind)
    torch.cuda.synchronize()
    assert r["status"] == [0, 0, 0] and r["scorer_status"] == 0 and len(lines) == 4
    # The draws are the 64-bit draws from the cycle's own logits.
    for logits, noise, tokens in zip(r["logits"], r["gumbel"], r["tokens"]):
        assert bool(torch.isfinite(logits).all())
        tokens, compared = tokens.reshape(-1).tolist(), 0
        for x in range(logits.shape[0]):
            want, _, margin = O.sample(logits[x], noise[x], 0.8, 40, 0.95, 0.02)
            if margin > 1e-4:
                compared += 1
                assert tokens[x] == want
        assert compared > logits.shape[0] // 2
    # The scores are those of the chain's logits.
    U, s = 2.0 ** -24, r["scores"]
    for x in range(r["given"].numel()):
        lp, rank, entropy, lse, ids, lps = P.scores(r["logits"][0][x], int(r["given"][x]), 0.8, 4)
        assert int(s.rank[x]) == rank and torch.equal(s.top_ids[x], ids)
        for got, want in ((s.logprob[x], lp), (s.entropy[x], entropy), (s.lse[x], lse)):
            assert abs(float(got) - want) <= 1000 * U + 4 * U * abs(want)
        assert bool(((s.top_logprob[x].double() - lps).abs() <= 1000 * U + 4 * U * lps.abs()).all())


def test_pages_in_the_layers_type_change_nothing():
    """bf16 pages hold what the cache in one piece holds: the cycle's logits and tokens are the same."""
    import target_cycle as T
    whole, pages = (T.main(log=lambda *a: None, pages=kind) for kind in (None, torch.bfloat16))
    for a, b in zip(whole["logits"], pages["logits"]):
        # One rounding of the layer's output each, 2^-8 of a logit's terms, where the kernels' sums differ in their last bits.
        assert float((a - b).abs().max()) <= 2.0 ** -7 * float(a.abs().max())
    assert torch.equal(whole["target"].ctx, pages["target"].ctx)
    for x, y in zip(whole["tokens"], pages["tokens"]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", KINDS)
def test_a_trees_logits_are_those_of_its_paths(kind):
    """Each node's path from the root as a causal block over the same past gives the tree's logits at its end."""
    import target_cycle as T
    r = T.main(log=lambda *a: None, pages=kind)
    target, (token, parent, depth) = r["target"], r["tree"]
    batch, rows = token.shape
    past = target.ctx - r["drafter"].advanced
    tree_logits = r["logits"][1].view(batch, rows, -1)
    pools = [p for p in (target.k, target.v, target.attn.k_scale, target.attn.v_scale) if p is not None]
    before = [p.view(torch.uint8).clone() for p in pools]
    target.ctx = past
    for node in range(rows):
        paths = []
        for b in range(batch):
            p, n = [], node
            while n >= 0:
                p.append(int(token[b, n]))
                n = int(parent[b, n])
            paths.append(p[::-1])
        start = torch.tensor([0] + [len(p) for p in paths], device="cuda").cumsum(0).to(torch.int32)
        h = target.hidden(torch.tensor(sum(paths, []), dtype=torch.int32, device="cuda"), q_start=start)
        last = h[(start[1:] - 1).long()].float() @ target.w["w_lm"].float().T
        for b in range(batch):
            # bf16 rows: two roundings of the layer's output apart, 2^-7 of a logit's terms
            bound = 2.0 ** -7 * float((h[start[b + 1] - 1].float().abs() @ target.w["w_lm"].float().abs().T).max())
            assert float((last[b] - tree_logits[b, node]).abs().max()) <= bound
        for p, was in zip(pools, before):
            p.view(torch.uint8).copy_(was)
