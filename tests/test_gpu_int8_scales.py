"""8-bit products whose scales multiply to less than the smallest normal binary32 number, or to more than the
largest: the result is that of the three factors together."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _codes(rows, cols, seed, low=-127):
    t = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.int8)
    t[:, :cols] = torch.randint(low, 128, (rows, cols), generator=torch.Generator().manual_seed(seed), dtype=torch.int8)
    return t.cuda()[:, :cols]


def _check(got, a, sa, b, sb, bias):
    torch.cuda.synchronize()
    ref = ops_ref.int8_product(*(t.cpu().numpy() for t in (a, sa, b, sb)), None if bias is None else bias.cpu().numpy())
    ops_ref.check_product(got, *ref)


# a token, few columns, small and middle tiles, the largest; row scales down to 2^-126 and the smallest of all
@pytest.mark.parametrize("M,N,K", [(1, 70, 5000), (5, 40, 300), (64, 100, 2048), (130, 260, 1000), (777, 1003, 515),
                                   (2100, 2310, 400), (2050, 6900, 300)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_of_small_scales(M, N, K, dtype):
    print(f"small scales M={M} N={N} K={K} {dtype}", flush=True)
    # sums far from 0, so that the results are normal numbers
    a, b = _codes(M, K, 1, low=60), _codes(N, K, 2, low=60)
    g = torch.Generator().manual_seed(3)
    for lowest, channel in ((2.0 ** -126, 1e-4), (2.0 ** -126, 1e-6), (2.0 ** -118, 1e-8), (2.0 ** -140, 1.0)):
        sa = (lowest * torch.exp(3.0 * torch.rand(M, generator=g))).cuda()
        sa[M // 2] = 0.01  # ordinary rows beside them
        sb = (channel * torch.exp(0.3 * torch.randn(N, generator=g))).cuda()
        for bias in (None, (2.0 ** -110 * torch.randn(N, generator=g)).cuda()):
            got = binding.int8_matmul(a, sa, b, sb, bias=bias, out_dtype=dtype)
            _check(got, a, sa, b, sb, bias)


@pytest.mark.parametrize("M,N,K", [(1, 70, 500), (5, 40, 300), (130, 260, 1000), (2100, 2310, 400)])
def test_product_of_large_scales(M, N, K):
    """A sum of 0 stays 0 where the scales alone overflow; the scales' order does not matter."""
    print(f"large scales M={M} N={N} K={K}", flush=True)
    a, b = _codes(M, K, 1), _codes(N, K, 2)
    a[M // 2] = 0
    sa, sb = torch.full((M,), 1e-9, device="cuda"), torch.full((N,), 1e3, device="cuda")
    sa[M // 2] = 1e36
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).cuda()
    got = binding.int8_matmul(a, sa, b, sb, bias=bias, out_dtype=F32)
    _check(got, a, sa, b, sb, bias)
    # the largest row scale there is, and a channel scale that brings the result back
    sa.fill_(2.6e36)
    sb.fill_(1e-12)
    _check(binding.int8_matmul(a, sa, b, sb, out_dtype=F32), a, sa, b, sb, None)


@pytest.mark.parametrize("M", [1, 2, 7, 16, 100, 700])
def test_linear_of_small_rows(M):
    """Rows whose largest value is a little above 2^-119, quantized in the product's kernel or before it."""
    K, N = 640, 200
    g = torch.Generator().manual_seed(M)
    x = (2.0 ** -118 * (1.0 + torch.rand((M, K), generator=g))).cuda()
    w = _codes(N, K, 2, low=60)
    for channel in (1e-4, 1e-6):
        sb = torch.full((N,), channel, device="cuda")
        got = binding.int8_linear(x, w, sb)
        torch.cuda.synchronize()
        ops_ref.check_product(got, *ops_ref.int8_product(*ops_ref.int8_rows(x), w.cpu().numpy(), sb.cpu().numpy()))
        q, s = binding.int8_quantize_per_token(x)
        assert torch.equal(got, binding.int8_matmul(q, s, w, sb, out_dtype=F32))
