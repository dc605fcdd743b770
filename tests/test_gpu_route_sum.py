"""Softmax weights over all experts (no renormalization, no bias): rounded once, as every other weight."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [8, 100, 160, 256, 300, 432, 512, 1000])
@pytest.mark.parametrize("T", [60, 2100])
@pytest.mark.parametrize("spread,shift", [(0.01, 0.0), (1.5, 0.0), (3.0, 40.0)])
def test_softmax_weights_are_rounded_once(E, T, spread, shift):
    print(f"route sum E={E} T={T} spread={spread}", flush=True)
    l = (spread * torch.randn((T, E), generator=torch.Generator().manual_seed(E)) + shift).cuda()
    ids, w = binding.route(l, min(E, 7), binding.Router(renormalize=False, scale=2.5))
    torch.cuda.synchronize()
    some = slice(None, None, 1 if T < 100 else 31)
    rids, rw = ops_ref.route(l[some], min(E, 7), renormalize=False, scale=2.5)
    np.testing.assert_array_equal(ids[some].cpu().numpy(), rids)
    # half a step of binary32, and the 2^-42 of the binary64 sum
    np.testing.assert_allclose(w[some].double().cpu().numpy(), rw, rtol=1.01 * 2.0 ** -24)
