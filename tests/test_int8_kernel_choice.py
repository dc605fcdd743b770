"""The 8-bit product's choice of a kernel can be asked on the host."""
import ctypes

from nvfp4_token_quant_amd import binding
from tests.test_gpu_operator_paths import PRODUCTS


def _kernel(M, N, K, lda=None, ldb=None):
    n, ld = ctypes.c_int32(-1), (K + 15) // 16 * 16
    status = binding.lib().int8_matmul_kernel(M, N, K, ld if lda is None else lda, ld if ldb is None else ldb,
                                              ctypes.byref(n))
    return n.value if status == 0 else -status


def test_every_kernel_is_tested():
    assert set(PRODUCTS) == set(range(9))
    for kernel, sizes in PRODUCTS.items():
        for size in sizes:
            assert _kernel(*size) == kernel, size
        # an end of K inside a step and inside 16 bytes, odd M and N
        assert any(K % 16 for _, _, K in sizes) and any(M % 16 for M, _, _ in sizes) and any(N % 16 for _, N, _ in sizes)


def test_limits():
    assert _kernel(1, 10, 32768) == 0 and _kernel(1, 10, 32769) > 0
    assert _kernel(500, 500, 64, lda=(1 << 22) + 16) == 2 and _kernel(500, 500, 64, ldb=1 << 26) == 2
    assert _kernel(2 ** 31 - 513, 1, 16) > 0 and _kernel(2 ** 31 - 512, 1, 16) == -1
    assert _kernel(1, 2 ** 31 - 512, 16) == -1
    for bad in ((0, 4, 16), (4, 0, 16), (-1, 4, 16), (4, 4, 0), (4, 4, 131072), (4, 4, 16, 8), (4, 4, 16, 24),
                (4, 4, 16, (1 << 26) + 16)):
        assert _kernel(*bad) == -1, bad
    assert binding.lib().int8_matmul_kernel(4, 4, 16, 16, 16, None) == 1
