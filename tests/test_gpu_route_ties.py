"""Routing ties: equal experts and equal groups go to the lower index, whatever lanes hold them, and a
token's routing does not depend on the batch that it comes with."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu


def _coarse(T, E, dtype, seed=0, step=0.5):
    """Logits of a coarse grid: every token has many experts of equal logits."""
    g = torch.Generator().manual_seed(seed)
    return (step * torch.randint(-4, 5, (T, E), generator=g)).to(dtype).cuda()


# 16 lanes a token, a wave by register swaps, a wave by shuffles; whole lanes a group or not
@pytest.mark.parametrize("T,E,groups,top_groups", [
    (700, 96, 8, 4), (300, 256, 8, 4), (2100, 256, 8, 4), (300, 300, 6, 3), (2100, 300, 10, 5), (2100, 384, 8, 4),
    (300, 512, 8, 4), (2100, 512, 8, 4), (300, 1000, 8, 4), (2060, 1000, 4, 2)])
@pytest.mark.parametrize("best", [0, 1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_softmax_with_a_bias_keeps_ties(T, E, groups, top_groups, best, dtype):
    print(f"route ties T={T} E={E} groups={groups}/{top_groups}/{best} {dtype}", flush=True)
    rule = dict(groups=groups, top_groups=top_groups, group_best=best) if best else {}
    l = _coarse(T, E, dtype, seed=E + best)
    for value in (0.0, 0.5, -0.375):
        b = torch.full((E,), value, device="cuda")
        ids, _ = binding.route(l, 8, binding.Router(**rule), bias=b)
        rids, _ = ops_ref.route(l, 8, bias=b, **rule)
        np.testing.assert_array_equal(ids.cpu().numpy(), rids)


@pytest.mark.parametrize("E,groups,top_groups", [(64, 8, 4), (160, 8, 4), (256, 8, 4), (300, 6, 3), (432, 3, 2),
                                                 (512, 8, 4), (1000, 8, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_routing_does_not_depend_on_the_batch(E, groups, top_groups, score, bias, renormalize):
    """Ids and weights of the first tokens are the same bit for bit in batches of any size."""
    print(f"route batches E={E} {score} bias={bias} renormalize={renormalize}", flush=True)
    g = torch.Generator().manual_seed(E)
    l = (1.5 * torch.randn((4100, E), generator=g)).cuda()
    b = (0.02 * torch.randn(E, generator=g)).cuda() if bias else None
    for rule in (dict(), dict(groups=groups, top_groups=top_groups, group_best=2)):
        r = binding.Router(score=score, renormalize=renormalize, **rule)
        ids, w = binding.route(l, 8, r, bias=b)
        for T in (1, 3, 200, 2048, 2049):
            part = binding.route(l[:T], 8, r, bias=b)
            assert torch.equal(part[0], ids[:T]), T
            assert torch.equal(part[1], w[:T]), T
