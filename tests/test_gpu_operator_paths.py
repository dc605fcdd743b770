"""Sizes that take the operators' less common paths: every tile of the 8-bit product, a block's second tile of
few tokens, wide and in-place norms, large batches of narrow norms, 16-bit logits of many experts; norms against a
tolerance for their own width."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed)) + shift).to(dtype).cuda()


def _codes(rows, cols, seed):
    ld = (cols + 15) // 16 * 16
    t = torch.randint(-128, 128, (rows, ld), generator=torch.Generator().manual_seed(seed), dtype=torch.int8)
    return t.cuda()[:, :cols]


def _kernel(M, N, K):
    n, ld = ctypes.c_int32(), (K + 15) // 16 * 16
    assert binding.lib().int8_matmul_kernel(M, N, K, ld, ld, ctypes.byref(n)) == 0
    return n.value


# each tile with whole and odd sizes, an odd and an even number of 128-byte steps, ends of K inside 16 bytes
PRODUCTS = {
    0: [(1, 129, 1000), (1, 4097, 333)],
    1: [(64, 100, 2048), (17, 97, 1337), (130, 260, 1000)],
    2: [(5, 40, 300), (100, 700, 2001), (129, 700, 1920)],
    3: [(300, 768, 2048), (259, 801, 1001), (259, 801, 2001), (257, 799, 2177)],
    4: [(300, 900, 1500), (333, 901, 1537)],
    5: [(777, 1003, 515), (513, 2049, 1500), (500, 2050, 1665)],
    6: [(777, 3001, 4001), (1000, 3000, 4096), (777, 3003, 3969), (300, 7168, 4111)],
    7: [(2100, 2310, 400), (600, 1900, 1111), (333, 5000, 260)],
    8: [(2050, 6900, 300), (2060, 6901, 256), (2050, 6903, 513)],
}


@pytest.mark.parametrize("kernel,M,N,K", [(k, *s) for k, sizes in PRODUCTS.items() for s in sizes])
def test_every_product_kernel(kernel, M, N, K):
    print(f"product kernel {kernel} M={M} N={N} K={K}", flush=True)
    assert _kernel(M, N, K) == kernel
    a, b = _codes(M, K, 1), _codes(N, K, 2)
    sa, sb = (1e-4 * torch.exp(0.5 * _randn(n, seed=n)) for n in (M, N))
    for dtype, bias in ((BF16, None), (F32, _randn(N, seed=5))):
        out = torch.full((M + 1, N + 3), -7.0, dtype=dtype, device="cuda")
        got = binding.int8_matmul(a, sa, b, sb, bias=bias, out=out[:M, 1:N + 1])
        torch.cuda.synchronize()
        ops_ref.check_product(got, *ops_ref.int8_product(*(t.cpu().numpy() for t in (a, sa, b, sb)),
                                                         None if bias is None else bias.cpu().numpy()))
        got.fill_(-7.0)
        assert (out == -7.0).all()  # nothing beside it
    # the first tokens alone, in the kernels of smaller batches, bit for bit
    whole = binding.int8_matmul(a, sa, b, sb, out_dtype=F32)
    for n in (1, 9, 40):
        assert torch.equal(binding.int8_matmul(a[:n], sa[:n], b, sb, out_dtype=F32), whole[:n])


@pytest.mark.parametrize("M,N,K", [(2, 8193, 1000), (2, 20001, 8192), (5, 8193, 130), (5, 20001, 2048), (16, 8208, 1024),
                                   (16, 20001, 600), (9, 16385, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens_of_many_channels(M, N, K, dtype):
    """Blocks of the one-kernel form that take more than one tile."""
    print(f"few tokens M={M} N={N} K={K} {dtype}", flush=True)
    x, w, ws = _randn(M, K, seed=1, dtype=dtype), _codes(N, K, 2), 1e-3 * torch.exp(0.5 * _randn(N, seed=3))
    bias = _randn(N, seed=4)
    got = binding.int8_linear(x, w, ws, bias=bias, out_dtype=F32)
    two = binding.int8_matmul(*binding.int8_quantize_per_token(x), w, ws, bias=bias, out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(got, two)
    ops_ref.check_product(got, *ops_ref.int8_product(*ops_ref.int8_rows(x), w.cpu().numpy(), ws.cpu().numpy(),
                                                     bias.cpu().numpy()))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("E,groups,top_groups", [(150, 3, 2), (192, 8, 4), (256, 8, 4), (300, 6, 3), (432, 4, 2), (510, 6, 3),
                                                 (1000, 8, 4)])
@pytest.mark.parametrize("T", [33, 2060])
def test_route_types_of_many_experts(E, groups, top_groups, T, dtype):
    """Wide loads of 4 to 32 logits a lane of each type, rows of any alignment."""
    print(f"route E={E} T={T} {dtype}", flush=True)
    l = _randn(T, E + 5, seed=E, dtype=dtype, scale=1.5)
    for c0 in (0, 3):
        v = l[:, c0:c0 + E]
        for bias, rule in ((None, dict()), (_randn(E, seed=9, scale=0.2), dict(score="sigmoid", groups=groups,
                                                                               top_groups=top_groups, group_best=2))):
            ids, w = binding.route(v, 9, binding.Router(**rule), bias=bias)
            torch.cuda.synchronize()
            some = slice(None, None, 1 if T < 100 else 29)  # (the reference goes token by token)
            rids, rw = ops_ref.route(v[some], 9, bias=bias, **rule)
            np.testing.assert_array_equal(ids[some].cpu().numpy(), rids)
            np.testing.assert_allclose(w[some].double().cpu().numpy(), rw, rtol=1.01 * 2.0 ** -24, atol=2.0 ** -150)


def _norm(H, dtype, kind, seed, bias):
    w, b = _randn(H, seed=seed, dtype=dtype, scale=0.3, shift=1.0), _randn(H, seed=seed + 1, dtype=dtype, scale=0.2)
    return (binding.Norm(w, b if bias else None, kind=kind),
            (ops_ref.f64(w), ops_ref.f64(b) if bias else None, kind, 1e-6, 0.0))


def _check_norm(r, y, after, before, gate, **kw):
    rr, rs, rh, hs = ops_ref.block_norm(r, y, before=before[1], after=after[1], gate=gate)
    got = binding.block_norm(r, y, before=before[0], after=after[0], gate=gate, **kw)
    torch.cuda.synchronize()
    ops_ref.check_norm(got[0], rr, rs)
    ops_ref.check_norm(got[1], rh, hs)
    return got


@pytest.mark.parametrize("H", [513, 520, 1001, 1024])
@pytest.mark.parametrize("T", [2049, 3001])
@pytest.mark.parametrize("dtype,residual", [(BF16, BF16), (BF16, F32), (F16, F32), (F32, F32)])
def test_norm_large_batches_of_narrow_rows(H, T, dtype, residual):
    """A wave takes a row of up to 1024 columns by itself."""
    print(f"norm T={T} H={H} {dtype} {residual}", flush=True)
    r, y = _randn(T, H, seed=1, dtype=residual, scale=2.0), _randn(T, H, seed=2, dtype=dtype)
    _check_norm(r, y, _norm(H, dtype, "layer", 3, True), _norm(H, dtype, "rms", 5, False),
                _randn(T, H, seed=7, dtype=dtype))


@pytest.mark.parametrize("H", [8200, 16385, 16400, 32768, 40000, 65535, 65536])
@pytest.mark.parametrize("dtype,residual", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_norm_wide_in_place(H, dtype, residual):
    """Rows whose residual and gate are read late, with an element gate, and in place."""
    print(f"norm in place H={H} {dtype} {residual}", flush=True)
    T = 3
    n1, n2 = _norm(H, dtype, "rms", 3, False), _norm(H, dtype, "layer", 5, True)
    big_r, big_y = _randn(T, H + 24, seed=1, dtype=residual), _randn(T, H + 40, seed=2, dtype=dtype)
    g = _randn(T, H + 8, seed=7, dtype=dtype)[:, 8:]
    for c0 in (0, 5):
        r, y = big_r[:, c0:c0 + H], big_y[:, c0:c0 + H]
        want = _check_norm(r, y, n1, n2, g)
        r2, y2 = big_r.clone(), big_y.clone()
        got = binding.block_norm(r2[:, c0:c0 + H], y2[:, c0:c0 + H], before=n2[0], after=n1[0], gate=g,
                                 residual_out=r2[:, c0:c0 + H], h_out=y2[:, c0:c0 + H])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for a, b in ((r2, big_r), (y2, big_y)):  # columns beside it stay as they were
            assert torch.equal(a[:, :c0], b[:, :c0]) and torch.equal(a[:, c0 + H:], b[:, c0 + H:])


def _chain(H):
    """The longest chain of additions of a row's sum: a thread's columns, six steps over a wave, its waves."""
    threads = 64 if H <= 512 else 128 if H <= 1024 else 256 if H <= 2048 else 512 if H <= 4096 else 1024
    return 8 * -(-H // (8 * threads)) + 1 + 6 + threads // 64


@pytest.mark.parametrize("H", [64, 512, 1000, 2048, 4096, 7168, 16384, 65536])
def test_norm_to_the_tolerance_of_its_width(H):
    """A norm in binary32 alone, u = 2^-24 a rounding.

    RMS: the squares' sum has positive terms, so it is off by at most its chain
    plus the squares' own rounding, (chain + 1) u; times 1 / cols (2 u: that
    number and the product) and plus eps (u), then half of all that under the
    root; the root, the quotient, weight times it and the product with the
    value: 4 u.
    Layer: the mean is off by (chain + 2) u of the mean magnitude, which every
    difference takes (and the squares' sum in second order: one more u), and a
    difference is rounded once, u of its own size, which its square doubles and
    the root halves."""
    T, u, n = 7, 2.0 ** -24, _chain(H)
    r, w = _randn(T, H, seed=1, shift=0.5), _randn(H, seed=2, scale=0.3, shift=1.0)
    r64, w64 = ops_ref.f64(r), ops_ref.f64(w)
    _, h = binding.block_norm(r, before=binding.Norm(w))
    want = r64 / np.sqrt((r64 ** 2).mean(1, keepdims=True) + 1e-6) * w64
    tol = ((n + 4) / 2 + 4) * u * np.abs(want)
    assert (np.abs(ops_ref.f64(h) - want) <= 1.001 * tol).all()
    _, h = binding.block_norm(r, before=binding.Norm(w, kind="layer"))
    d = r64 - r64.mean(1, keepdims=True)
    inv = 1.0 / np.sqrt((d ** 2).mean(1, keepdims=True) + 1e-6)
    tol = ((n + 4) / 2 + 7) * u * np.abs(d * inv * w64) \
        + (n + 2) * u * np.abs(r64).mean(1, keepdims=True) * inv * np.abs(w64)
    assert (np.abs(ops_ref.f64(h) - d * inv * w64) <= 1.001 * tol).all()
