"""8-bit quantization (bit for bit) and products (exact sums) against the CPU."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check_quant(x, **kw):
    q, s = binding.int8_quantize_per_token(x, **kw)
    torch.cuda.synchronize()
    rq, rs = ops_ref.int8_rows(x)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    return q, s


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cols", [1, 7, 8, 15, 16, 24, 512, 513, 1000, 1024, 1999, 2048, 4096, 4104, 7168, 8192, 9000,
                                  16384, 16392, 20001, 40000])
def test_quantize_widths(dtype, cols):
    print(f"int8 quantize cols={cols} {dtype}", flush=True)
    rows = 9 if cols < 10000 else 3
    x = _randn(rows, cols, seed=cols, dtype=dtype)
    x[1] = 0.0
    x[2, cols // 2] = 37.0
    _check_quant(x)
    # zeros behind cols up to a whole 16-byte piece
    full = binding.int8_quantize_per_token(x)[0]
    pad = full.as_strided((rows, (cols + 15) // 16 * 16), ((cols + 15) // 16 * 16, 1))[:, cols:]
    assert not pad.any()


def test_quantize_edges():
    x = torch.zeros((8, 64), device="cuda")
    x[0, 3] = 2.0 ** -119
    x[1, 3] = 2.0 ** -120
    x[2, 3] = torch.finfo(F32).tiny / 4
    x[3] = torch.finfo(F32).max
    x[4] = -torch.finfo(F32).max
    x[5] = torch.arange(64) - 31.5
    x[6, 0], x[6, 1] = 254.0, 127.0     # half of the largest: 63.5 up to rounding
    x[7, 0], x[7, 1] = -3.0, 1.5
    _check_quant(x)
    big = _randn(40, 96, seed=1, dtype=BF16)
    for v in (big[:, 8:72], big[::3], big[:, 3:50], big[5:6, 1:]):
        _check_quant(v)
    q, s = binding.int8_quantize_per_token(big[:0])
    assert q.shape == (0, 96) and s.shape == (0,)


def _codes(rows, cols, seed, full_range=False):
    g = torch.Generator().manual_seed(seed)
    ld = (cols + 15) // 16 * 16
    # bytes behind cols have no effect: anything
    t = torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int8).cuda()
    if full_range:
        t.fill_(-128)
    return t[:, :cols]


def _scales(n, seed):
    return (0.01 * torch.exp(0.5 * torch.randn(n, generator=torch.Generator().manual_seed(seed)))).cuda()


def _check_product(a, sa, b, sb, bias=None, dtype=BF16, **kw):
    got = binding.int8_matmul(a, sa, b, sb, bias=bias, out_dtype=dtype, **kw)
    torch.cuda.synchronize()
    ref = ops_ref.int8_product(*(t.cpu().numpy() for t in (a, sa, b, sb)), bias.cpu().numpy() if bias is not None else None)
    ops_ref.check_product(got, *ref)
    return got


SIZES = [(1, 1, 1), (1, 16, 64), (1, 300, 7168), (2, 17, 100), (3, 2048, 256), (5, 64, 131071), (16, 16, 128), (17, 33, 65),
         (31, 100, 1999), (40, 256, 2048), (64, 512, 1024), (65, 130, 513), (100, 1003, 777), (128, 128, 128),
         (129, 257, 300), (200, 512, 640), (255, 255, 255), (256, 256, 256), (257, 1030, 1111), (300, 768, 2048),
         (513, 1024, 384), (777, 1003, 1999), (1024, 512, 1024), (1030, 2050, 128), (2100, 384, 272),
         # every tile shape of the kernel, one to a few steps of K, whole and partial
         (90, 1100, 300), (150, 1900, 131), (300, 1001, 400), (500, 1033, 200), (1000, 3001, 129), (2050, 3000, 260),
         (1111, 5999, 100), (2060, 6900, 100), (2060, 6901, 256), (2050, 6900, 300), (2100, 6904, 388)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_sizes(M, N, K):
    print(f"int8 product M={M} N={N} K={K}", flush=True)
    a, b, sa, sb = _codes(M, K, 1), _codes(N, K, 2), 0.01 * _scales(M, 3), 0.01 * _scales(N, 4)
    _check_product(a, sa, b, sb, dtype=BF16)
    _check_product(a, sa, b, sb, bias=_randn(N, seed=5), dtype=F32)
    _check_product(a, sa, b, sb, bias=_randn(N, seed=5), dtype=F16)


def test_product_does_not_depend_on_the_batch():
    """A token's result is the same bit for bit in every batch, and so in every kernel."""
    K, N = 333, 900
    a, sa, b, sb = _codes(2600, K, 1), _scales(2600, 3), _codes(N, K, 2), _scales(N, 4)
    bias = _randn(N, seed=5)
    whole = binding.int8_matmul(a, sa, b, sb, bias=bias, out_dtype=F32)
    for M in (1, 2, 17, 40, 100, 300, 700, 1300, 2000):
        assert torch.equal(binding.int8_matmul(a[:M], sa[:M], b, sb, bias=bias, out_dtype=F32), whole[:M]), M


@pytest.mark.parametrize("M", [2, 40, 300])
def test_product_full_range(M):
    """The largest sum that int32 holds: 131071 products of (-128)^2."""
    K = 131071
    a, b = _codes(M, K, 1, True), _codes(16, K, 2, True)
    one = torch.ones(300, device="cuda")
    got = binding.int8_matmul(a, one[:M], b, one[:16], out_dtype=F32)
    torch.cuda.synchronize()
    assert (got == float(np.float32(K * 16384))).all()


@pytest.mark.parametrize("M,N", [(1, 40), (8, 200), (50, 200), (300, 520)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_strides(M, N, dtype):
    """Rows further apart, columns inside a larger matrix, an output inside a larger one; a single row."""
    K = 200
    a, b = _codes(M + 1, 480, 1)[1:, 32:32 + K], _codes(2 * N, 336, 2)[::2, 16:16 + K]
    sa, sb = _scales(M, 3), _scales(N, 4)
    for c0 in (0, 8, 5):
        big = torch.full((M + 2, N + 16), -7.0, dtype=dtype, device="cuda")
        _check_product(a, sa, b, sb, out=big[1:M + 1, c0:c0 + N], bias=_randn(N, seed=5))
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:M + 1, c0:c0 + N] = False
        assert (big[keep] == -7.0).all()


def test_product_far_offsets():
    ld, M, N, K = 1 << 26, 70, 40, 96
    buf = torch.empty(((M - 1) * ld + K,), dtype=torch.int8, device="cuda")
    a = buf.as_strided((M, K), (ld, 1))
    a.copy_(_codes(M, K, 1))
    b = _codes(N, K, 2)
    _check_product(a, _scales(M, 3), b, _scales(N, 4))
    _check_product(b, _scales(N, 4), a, _scales(M, 3))
    out = torch.empty(((M - 1) * ld + N,), dtype=F16, device="cuda").as_strided((M, N), (ld, 1))
    _check_product(a, 0.01 * _scales(M, 3), b, 0.01 * _scales(N, 4), out=out)


@pytest.mark.parametrize("M,N,K,dtype", [(1, 500, 1000, BF16), (33, 256, 2048, F16), (400, 520, 1001, F32)])
def test_linear(M, N, K, dtype):
    x, w = _randn(M, K, seed=1, dtype=dtype), _randn(N, K, seed=2)
    wq, ws = binding.int8_quantize_per_token(w)
    bias = _randn(N, seed=3)
    got = binding.int8_linear(x, wq, ws, bias=bias)
    torch.cuda.synchronize()
    assert got.dtype == dtype
    ref = ops_ref.int8_product(*ops_ref.int8_rows(x), *ops_ref.int8_rows(w), bias.cpu().numpy())
    ops_ref.check_product(got, *ref)
    # and near the unquantized product: an element is off by at most half a code of each operand,
    # amax/254, so the sum by sum_k |x| w_amax/254 + |w| x_amax/254 + their product
    x64, w64 = ops_ref.f64(x), ops_ref.f64(w)
    ex, ew = np.abs(x64).max(1) / 254, np.abs(w64).max(1) / 254
    tol = np.abs(x64).sum(1)[:, None] * ew + ex[:, None] * np.abs(w64).sum(1) + K * ex[:, None] * ew
    full = x64 @ w64.T + ops_ref.f64(bias)
    assert (np.abs(ops_ref.f64(got) - full) <= 1.01 * tol + ops_ref.EPS[dtype] * np.abs(full)).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = binding.int8_linear(x, wq, ws, bias=bias, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other, got)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 9), (8, 1024), (2048, 7168), (5000, 640), (300, 8192), (100, 8193),
                                 (64, 20001), (40, 32768), (33, 32769), (16, 131071)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_linear_one_token(N, K, dtype):
    """One token in one kernel equals the two steps bit for bit, and the reference."""
    print(f"one token N={N} K={K} {dtype}", flush=True)
    for c0, seed in ((0, 1), (1, 2)):
        x = _randn(1, K + c0, seed=seed, dtype=dtype)[:, c0:]
        if seed == 2:
            x[0, K // 2] = -90.0
        w, ws = _codes(N, K, 3), 0.01 * _scales(N, 4)
        bias = _randn(N, seed=5)
        got = binding.int8_linear(x, w, ws, bias=bias, out_dtype=F32)
        q, s = binding.int8_quantize_per_token(x)
        two = binding.int8_matmul(q, s, w, ws, bias=bias, out_dtype=F32)
        torch.cuda.synchronize()
        assert torch.equal(got, two)
        ops_ref.check_product(got, *ops_ref.int8_product(*ops_ref.int8_rows(x), w.cpu().numpy(), ws.cpu().numpy(),
                                                         bias.cpu().numpy()))
    zero = binding.int8_linear(torch.zeros((1, K), dtype=dtype, device="cuda"), w, ws, bias=bias)
    torch.cuda.synchronize()
    assert torch.equal(zero, bias.to(dtype)[None])


@pytest.mark.parametrize("M,N,K", [(2, 1, 1), (2, 40, 8192), (2, 20, 8193), (3, 100, 4095), (4, 2048, 4096), (5, 33, 2048),
                                   (5, 30, 2049), (7, 4096, 130), (7, 4097, 130), (8, 500, 2047), (9, 64, 1024),
                                   (16, 4096, 1000), (16, 17, 127), (13, 4090, 640), (16, 24, 1025), (17, 24, 512), (49, 61, 70),
                                   (33, 500, 1024), (512, 256, 512), (513, 256, 512), (31, 33, 1023), (8191, 7, 20)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_linear_few_tokens(M, N, K, dtype):
    """Few tokens in one kernel (and the next larger sizes in two) equal the two steps bit for bit, and the reference."""
    print(f"few tokens M={M} N={N} K={K} {dtype}", flush=True)
    for c0, seed in ((0, 1), (1, 2)):
        x = _randn(M, K + c0, seed=seed, dtype=dtype)[:, c0:]
        x[M - 1, K // 2] = -90.0
        x[M // 2] = 0.0
        w, ws = _codes(N, K, 3), 0.01 * _scales(N, 4)
        bias = _randn(N, seed=5) if seed == 1 else None
        out = torch.full((M + 2, N + 3), 5.0, device="cuda")
        got = binding.int8_linear(x, w, ws, bias=bias, out=out[1:-1, 2:-1])
        q, s = binding.int8_quantize_per_token(x)
        two = binding.int8_matmul(q, s, w, ws, bias=bias, out_dtype=F32)
        torch.cuda.synchronize()
        assert torch.equal(got, two)
        ops_ref.check_product(got, *ops_ref.int8_product(*ops_ref.int8_rows(x), w.cpu().numpy(), ws.cpu().numpy(),
                                                         None if bias is None else bias.cpu().numpy()))
        got.fill_(5.0)
        assert (out == 5.0).all()  # what is beside it stays as it was
        assert torch.equal(binding.int8_linear(x, w, ws, bias=bias), two.to(dtype))


def test_product_refusals_and_empty():
    a, b, sa, sb = _codes(4, 64, 1), _codes(8, 64, 2), _scales(4, 3), _scales(8, 4)
    assert binding.int8_matmul(a[:0], sa[:0], b, sb).shape == (0, 8)
    assert binding.int8_matmul(a, sa, b[:0], sb[:0]).shape == (4, 0)
    odd = torch.zeros((4, 63), dtype=torch.int8, device="cuda")
    for args in ((odd, sa, b[:, :63], sb), (a, sa[:3], b, sb), (a, sa, b[:, :48], sb), (a.float(), sa, b, sb),
                 (a, sa.double(), b, sb)):
        with pytest.raises(ValueError):
            binding.int8_matmul(*args)
    with pytest.raises(ValueError):
        binding.int8_matmul(a, sa, b, sb, out_dtype=torch.float64)
    with pytest.raises(binding.Nvfp4Error):
        binding.int8_matmul(a[:, 8:40], sa, b[:, 8:40], sb)          # rows not 16-byte aligned


@pytest.mark.parametrize("M", [1, 6, 16, 48, 600])
def test_linear_graph_replay(M):
    x = _randn(M, 1024, seed=1, dtype=BF16)
    wq, ws = binding.int8_quantize_per_token(_randn(520, 1024, seed=2))
    out = binding.int8_linear(x, wq, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            binding.int8_linear(x, wq, ws, out=out)
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(_randn(M, 1024, seed=10 + i))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, binding.int8_linear(x, wq, ws))


def test_rows_past_one_grid_dimension():
    """More rows than a launch has blocks in x: quantization and product of 2^21 + 3 and 2^25 + 40 tokens."""
    x = torch.zeros(((1 << 21) + 3, 600), dtype=BF16, device="cuda")
    x[-4:] = _randn(4, 600, seed=1, dtype=BF16)
    q, s = binding.int8_quantize_per_token(x)
    torch.cuda.synchronize()
    rq, rs = ops_ref.int8_rows(x[-4:])
    np.testing.assert_array_equal(q[-4:].cpu().numpy(), rq)
    np.testing.assert_array_equal(s[-4:].cpu().numpy(), rs)
    del x, q, s
    M = (1 << 25) + 40
    a = torch.zeros((M, 16), dtype=torch.int8, device="cuda")
    a[-50:] = _codes(50, 16, 1)
    sa = torch.ones(M, device="cuda")
    b, sb = _codes(8, 16, 2), _scales(8, 4)
    got = binding.int8_matmul(a, sa, b, sb, out_dtype=F32)
    torch.cuda.synchronize()
    ops_ref.check_product(got[-50:], *ops_ref.int8_product(a[-50:].cpu().numpy(), np.ones(50), b.cpu().numpy(),
                                                           sb.cpu().numpy()))
    assert not got[:-50].any()
