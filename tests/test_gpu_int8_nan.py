"""A row of activations with an infinity or a NaN: its products are NaN, all of them, and no other row's change."""
import pytest
import torch

from nvfp4_token_quant_amd import binding, synth
from nvfp4_token_quant_amd.block import MoeBlock
from tests.layer_fixtures import gpu_weights

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BROKEN = (float("nan"), float("inf"), -float("inf"), -float("nan"))


def _rows(M, K, dtype, seed=1):
    """Finite rows, the same with broken values in some, and which those are."""
    good = torch.randn((M, K), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    x, bad = good.clone(), torch.zeros(M, dtype=torch.bool, device="cuda")
    for i, v in enumerate(BROKEN):
        r = (2 * i + (M > 1)) % M
        x[r, (K - 1) * i // (len(BROKEN) - 1)] = v
        bad[r] = True
    return good, x, bad


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (9, 40), (9, 512), (9, 1000), (9, 2048), (9, 4096), (9, 8191), (9, 16384),
                                 (9, 20001)])
def test_quantize_keeps_broken_rows(M, K, dtype):
    print(f"broken rows M={M} K={K} {dtype}", flush=True)
    good, x, bad = _rows(M, K, dtype)
    want_q, want_s = binding.int8_quantize_per_token(good)
    q, s = binding.int8_quantize_per_token(x)
    torch.cuda.synchronize()
    assert torch.isnan(s[bad]).all()
    assert torch.equal(s[~bad], want_s[~bad]) and torch.equal(q[~bad], want_q[~bad])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 70, 1000), (1, 70, 20000), (9, 70, 1000), (4, 70, 4000), (2, 70, 8000), (40, 70, 600),
                                   (40, 300, 2000), (300, 520, 1001)])
def test_linear_keeps_broken_rows(M, N, K, dtype):
    print(f"broken rows M={M} N={N} K={K} {dtype}", flush=True)
    good, x, bad = _rows(M, K, dtype)
    w, ws = binding.int8_quantize_per_token(torch.randn((N, K), generator=torch.Generator().manual_seed(2)).cuda())
    for bias in (None, torch.ones(N, device="cuda")):
        want = binding.int8_linear(good, w, ws, bias=bias)
        got = binding.int8_linear(x, w, ws, bias=bias)
        torch.cuda.synchronize()
        assert torch.isnan(got[bad]).all()
        assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("T", [6, 100])
@pytest.mark.parametrize("score", [None, "sigmoid"])
def test_block_keeps_a_broken_row_to_itself(T, score):
    """A NaN in one token's residual: its router logits are NaN, its output is NaN, and no other token's changes."""
    print(f"block with a broken row T={T} router {score}", flush=True)
    L = synth.LAYERS[1]
    g = torch.Generator().manual_seed(T)
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(1))
    if score:
        layer.set_router(binding.Router(score=score, groups=4, top_groups=2))
    wg, sg = binding.int8_quantize_per_token((torch.randn((L.E, L.H), generator=g) * L.H ** -0.5).cuda())
    n = binding.Norm((1 + 0.2 * torch.randn(L.H, generator=g)).to(BF16).cuda())
    block = MoeBlock(layer, wg, sg, n)
    r = torch.randn((T, L.H), generator=g).to(BF16).cuda()
    want, wh = block.forward(r, next_before=n)
    r[T // 2, 3] = float("nan")
    got, gh = block.forward(r, next_before=n)
    torch.cuda.synchronize()
    rest = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(got[rest], want[rest]) and torch.equal(gh[rest], wh[rest])
    assert torch.isnan(got[T // 2, 3]) and torch.isnan(gh[T // 2]).all()
    layer.close()
