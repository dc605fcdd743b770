"""Argument checks of the operators around the layer (no GPU needed): each
refusal returns its documented status before any device work; empty inputs
are no-ops; the references that the GPU tests use are pinned on the CPU."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

P = ctypes.c_void_p
BF16, F16, F32 = 0, 1, 2


def _router(**kw):
    c = dict(score=0, num_groups=1, top_groups=1, group_best=1, renormalize=1, scale=1.0)
    c.update(kw)
    return binding.MoeRouter(**c)


def _route(r=None, logits=1 << 20, dtype=F32, T=4, E=16, ld=16, k=2, bias=0, ids=1 << 21, w=1 << 22):
    return binding.lib().moe_route(r if r is not None else _router(), P(logits), dtype, T, E, ld, k, P(bias), P(ids),
                                   P(w), None)


def test_route_refusals():
    for bad in (dict(score=2), dict(num_groups=0), dict(num_groups=3), dict(num_groups=65, top_groups=65),
                dict(num_groups=4, top_groups=5), dict(num_groups=4, top_groups=0), dict(group_best=0),
                dict(num_groups=4, top_groups=2, group_best=3), dict(renormalize=2), dict(scale=float("inf")),
                dict(scale=float("nan"))):
        assert _route(_router(**bad)) == 1, bad
    assert _route(_router(num_groups=8, top_groups=1), k=3) == 1        # one group of two experts
    assert binding.lib().moe_route(None, P(64), F32, 1, 8, 8, 2, None, P(128), P(256), None) == 1
    assert _route(E=0) == 1 and _route(E=1025, ld=1025) == 1
    assert _route(k=0) == 1 and _route(k=17, E=32, ld=32) == 1 and _route(k=9, E=8) == 1
    assert _route(dtype=3) == 1 and _route(ld=15) == 1 and _route(T=-1) == 1 and _route(T=2 ** 31) == 1
    assert _route(logits=0) == 1 and _route(ids=0) == 1 and _route(w=0) == 1
    assert _route(logits=(1 << 20) + 2) == 1 and _route(bias=2) == 1 and _route(ids=(1 << 21) + 1) == 1
    assert _route(ids=(1 << 20) + 64) == 3 and _route(w=(1 << 20) + 64) == 3   # inside the logits
    assert _route(ids=1 << 22, w=(1 << 22) + 16) == 3
    assert _route(bias=1 << 21) == 3
    assert _route(T=0, logits=0, ids=0, w=0) == 0


def test_set_router_refusals():
    assert binding.lib().moe_workspace_set_router(None, _router(), None, None) == 1


def _norm_args(**kw):
    c = dict(rows=4, cols=64, dtype=BF16, residual_dtype=BF16, residual=1 << 20, ld_residual=64, y=1 << 21, ld_y=64,
             gate=None, ld_gate=0, gate_cols=0, gate_sigmoid=0, res_scale=1.0, out_scale=1.0, residual_out=1 << 22,
             ld_residual_out=64, h=None, ld_h=0)
    after, before = kw.pop("after", None), kw.pop("before", None)
    c.update(kw)
    a = binding.MoeBlockNormArgs(**c)
    a.after = ctypes.pointer(after) if after is not None else None
    a.before = ctypes.pointer(before) if before is not None else None
    return binding.lib().moe_block_norm(ctypes.byref(a), None)


def test_block_norm_refusals():
    rms = binding.MoeNorm(0, 1e-6, 0.0, None, None)
    assert binding.lib().moe_block_norm(None, None) == 1
    for bad in (dict(dtype=3), dict(dtype=BF16, residual_dtype=F16), dict(dtype=F32, residual_dtype=BF16),
                dict(rows=-1), dict(rows=2 ** 31), dict(cols=0), dict(cols=65537), dict(ld_residual=63),
                dict(ld_y=63), dict(ld_residual_out=63), dict(y=None, after=rms), dict(y=None, gate=1 << 23),
                dict(h=1 << 23, ld_h=64), dict(before=rms), dict(h=1 << 23, ld_h=63, before=rms),
                dict(gate=1 << 23, gate_cols=2, ld_gate=0), dict(gate=1 << 23, gate_cols=64, ld_gate=63),
                dict(gate_sigmoid=2), dict(res_scale=float("nan")), dict(out_scale=float("inf")),
                dict(residual=None), dict(residual_out=None), dict(residual=(1 << 20) + 1), dict(y=(1 << 21) + 1),
                dict(gate=(1 << 23) + 1, gate_cols=64), dict(after=binding.MoeNorm(2, 1e-6, 0.0, None, None)),
                dict(after=binding.MoeNorm(0, -1.0, 0.0, None, None)),
                dict(after=binding.MoeNorm(0, float("nan"), 0.0, None, None)),
                dict(after=binding.MoeNorm(0, 1e-6, float("inf"), None, None)),
                dict(after=binding.MoeNorm(0, 1e-6, 0.0, 65, None))):
        assert _norm_args(**bad) == 1, bad
    hn = dict(h=1 << 23, ld_h=64, before=rms)
    for alias in (dict(residual_out=(1 << 20) + 64), dict(residual_out=1 << 20, ld_residual_out=128, ld_residual=64),
                  dict(residual_out=(1 << 21)), dict(hn, h=1 << 20), dict(hn, h=1 << 22), dict(hn, h=(1 << 21) + 64),
                  dict(gate=1 << 22, gate_cols=64, ld_gate=64),
                  dict(after=binding.MoeNorm(0, 1e-6, 0.0, 1 << 22, None))):
        assert _norm_args(**alias) == 3, alias
    assert _norm_args(rows=0, residual=None, y=None, residual_out=None) == 0


def _quant(x=1 << 20, dtype=BF16, rows=4, cols=40, ld=40, codes=1 << 21, ldc=48, scale=1 << 22):
    return binding.lib().int8_quantize_per_token(P(x), dtype, rows, cols, ld, P(codes), ldc, P(scale), None)


def _matmul(a=1 << 20, lda=64, sa=1 << 21, b=1 << 22, ldb=64, sb=1 << 23, bias=0, M=4, N=8, K=60, out=1 << 24, dtype=BF16,
            ldo=8):
    return binding.lib().int8_matmul(P(a), lda, P(sa), P(b), ldb, P(sb), P(bias), M, N, K, P(out), dtype, ldo, None)


def test_int8_refusals():
    assert _quant(dtype=5) == 1 and _quant(rows=-1) == 1 and _quant(cols=0) == 1 and _quant(ld=39) == 1
    assert _quant(ldc=40) == 1 and _quant(ldc=32) == 1 and _quant(x=0) == 1 and _quant(codes=0) == 1
    assert _quant(scale=0) == 1 and _quant(x=(1 << 20) + 1) == 1 and _quant(codes=(1 << 21) + 8) == 1
    assert _quant(codes=(1 << 20) + 64) == 3 and _quant(scale=(1 << 20) + 64) == 3 and _quant(scale=1 << 21) == 3
    assert _quant(rows=0, x=0) == 0
    assert _matmul(dtype=-1) == 1 and _matmul(M=-1) == 1 and _matmul(N=2 ** 31) == 1 and _matmul(K=0) == 1
    assert _matmul(K=131072, lda=131072, ldb=131072) == 1 and _matmul(lda=72) == 1 and _matmul(ldb=48) == 1
    assert _matmul(lda=(1 << 26) + 16) == 1 and _matmul(ldb=(1 << 26) + 16) == 1
    assert _matmul(ldo=7) == 1 and _matmul(a=0) == 1 and _matmul(sa=0) == 1 and _matmul(out=0) == 1
    assert _matmul(a=(1 << 20) + 8) == 1 and _matmul(b=(1 << 22) + 4) == 1 and _matmul(bias=2) == 1
    assert _matmul(out=(1 << 20) + 16) == 3 and _matmul(out=1 << 22) == 3 and _matmul(out=1 << 23) == 3
    assert _matmul(bias=1 << 24) == 3
    assert _matmul(M=0) == 0 and _matmul(N=0) == 0
    assert b"" == binding.lib().nvfp4_last_error()


def _linear(x=1 << 20, dtype=BF16, ldx=60, w=1 << 21, ldw=64, sw=1 << 22, bias=0, M=17, N=8, K=60, ws=1 << 23,
            wsb=17 * 68, out=1 << 24, odt=BF16, ldo=8):
    return binding.lib().int8_linear(P(x), dtype, ldx, P(w), ldw, P(sw), P(bias), M, N, K, P(ws), wsb, P(out), odt, ldo,
                                     None)


def test_int8_linear_refusals():
    n = ctypes.c_int64()
    assert binding.lib().int8_linear_workspace(17, 60, ctypes.byref(n)) == 0 and n.value == 17 * 68
    none = ((1, 1), (1, 32768), (2, 16), (2, 8192), (3, 4096), (4, 4096), (5, 2048), (8, 2048), (9, 1024), (16, 1024))
    for M, K in (*none, (0, 5), (1, 32769), (1, 131071), (2, 8193), (3, 4097), (5, 2049), (16, 1025), (17, 16), (300, 1001)):
        assert binding.lib().int8_linear_workspace(M, K, ctypes.byref(n)) == 0
        assert n.value == (0 if (M, K) in none else M * ((K + 15) // 16 * 16 + 4))
    assert binding.lib().int8_linear_workspace(4, 0, ctypes.byref(n)) == 1
    assert binding.lib().int8_linear_workspace(-1, 60, ctypes.byref(n)) == 1
    assert binding.lib().int8_linear_workspace(4, 60, None) == 1
    assert _linear(dtype=3) == 1 and _linear(odt=3) == 1 and _linear(ldx=59) == 1 and _linear(K=0) == 1
    assert _linear(ldw=60) == 1 and _linear(wsb=17 * 68 - 1) == 1 and _linear(ws=0) == 1 and _linear(ws=(1 << 23) + 8) == 1
    assert _linear(x=0) == 1 and _linear(w=0) == 1 and _linear(sw=0) == 1 and _linear(out=0) == 1 and _linear(M=-1) == 1
    for alias in (dict(out=1 << 20), dict(out=1 << 21), dict(out=1 << 22), dict(out=1 << 23), dict(ws=1 << 20),
                  dict(ws=1 << 21), dict(ws=1 << 22), dict(bias=1 << 23), dict(bias=1 << 24)):
        assert _linear(**alias) == 3, alias
    assert _linear(M=1, ws=0, wsb=0, x=0) == 1 and _linear(M=1, ws=0, wsb=0, out=1 << 20) == 3
    assert _linear(M=16, ws=0, wsb=0, x=0) == 1 and _linear(M=16, ws=0, wsb=0, out=1 << 20) == 3
    assert _linear(M=0, x=0, ws=0, wsb=0, out=0) == 0 and _linear(N=0, w=0, sw=0, out=0) == 0


def test_python_refusals():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        binding.route(x, 2, binding.Router())
    with pytest.raises(ValueError):
        binding.block_norm(x)
    with pytest.raises(ValueError):
        binding.int8_quantize_per_token(x)
    with pytest.raises(ValueError):
        binding.int8_matmul(x.to(torch.int8), x[:, 0], x.to(torch.int8), x[:, 0])
    with pytest.raises(ValueError):
        binding.int8_linear(x, x.to(torch.int8), x[:, 0])
    with pytest.raises(ValueError):
        binding.int8_quantize_per_token([[1.0]])
    with pytest.raises(TypeError):
        binding.route(x)
    with pytest.raises(ValueError):
        binding.Router(score="relu")
    with pytest.raises(ValueError):
        binding.Norm(kind="batch")


def test_route_reference_against_torch():
    g = torch.Generator().manual_seed(0)
    l = torch.randn((50, 24), generator=g, dtype=torch.float64)
    ids, w = ops_ref.route(l, 5)
    v, i = torch.topk(l, 5)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, torch.softmax(v, 1).numpy(), rtol=1e-12)
    ids, w = ops_ref.route(l, 5, renormalize=False, scale=2.0)
    np.testing.assert_allclose(w, 2 * torch.softmax(l, 1).gather(1, i).numpy(), rtol=1e-12)
    b = torch.randn(24, generator=g, dtype=torch.float64)
    ids, w = ops_ref.route(l, 5, "sigmoid", b, groups=6, top_groups=3, group_best=2)
    s = torch.sigmoid(l)
    v = s + b
    best = v.view(50, 6, 4).topk(2, dim=2).values.sum(2).topk(3, dim=1).indices
    keep = torch.zeros(50, 6, dtype=torch.bool).scatter_(1, best, True).repeat_interleave(4, 1)
    i = v.masked_fill(~keep, -torch.inf).topk(5).indices
    np.testing.assert_array_equal(ids, i.numpy())
    p = s.gather(1, i)
    np.testing.assert_allclose(w, (p / p.sum(1, keepdim=True)).numpy(), rtol=1e-12)
    ids, w = ops_ref.route(np.full((1, 8), -np.inf), 3, "sigmoid", groups=4, top_groups=2)
    assert ids.tolist() == [[0, 1, 2]] and not w.any()


def test_norm_reference_against_torch():
    g = torch.Generator().manual_seed(1)
    x, w, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((6, 40), (40,), (40,)))
    r, _, h, _ = ops_ref.block_norm(x, None, before=(w.numpy(), b.numpy(), "layer", 1e-5, 0.0))
    np.testing.assert_allclose(h, torch.nn.functional.layer_norm(x, (40,), w, b, 1e-5).numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_array_equal(r, x.numpy())
    _, _, h, _ = ops_ref.block_norm(x, None, before=(w.numpy(), None, "rms", 1e-5, 1.0))
    np.testing.assert_allclose(h, torch.nn.functional.rms_norm(x, (40,), w + 1, 1e-5).numpy(), rtol=1e-11)


def test_norm_check_catches_a_mistake_in_the_oracle():
    x = torch.randn((4, 64), generator=torch.Generator().manual_seed(2))
    r, rs, h, hs = ops_ref.block_norm(x, None, before=(np.ones(64), None, "rms", 1e-6, 0.0))
    ops_ref.check_norm(torch.from_numpy(h).float(), h, hs)
    bad = h.copy()
    bad[1, 3] *= 1.001
    with pytest.raises(AssertionError):
        ops_ref.check_norm(torch.from_numpy(h).float(), bad, hs)


def test_int8_reference_by_hand():
    # amax 127: scale 1, codes the nearest whole numbers, ties to even; a row below 2^-119 and a zero row
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5], [2.0 ** -120, 0.0, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0],
                      [4.0, 2.0, -1.0, 0.0]])
    q, s = ops_ref.int8_rows(x)
    assert q.tolist()[:3] == [[127, 0, 2, -2], [0, 0, 0, 0], [0, 0, 0, 0]]
    assert s.tolist()[:3] == [1.0, 1.0, 1.0]
    assert q[3].tolist() == [127, 64, -32, 0] and s[3] == np.float32(4.0) / np.float32(127.0)
    out, _ = ops_ref.int8_product(q[3:], s[3:], np.full((1, 4), 3, np.int8), np.ones(1, np.float32), np.ones(1, np.float32))
    np.testing.assert_allclose(out, [[(127 + 64 - 32) * 3 * float(s[3]) + 1]])
