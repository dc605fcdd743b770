"""Norms after and before a block, with gate and residual, against 64 bits."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed)) + shift).to(dtype).cuda()


def _make_norm(H, dtype, kind, offset, bias, seed, eps=1e-6, weight=True):
    w = _randn(H, seed=seed, dtype=dtype, scale=0.3, shift=1.0 - offset) if weight else None
    b = _randn(H, seed=seed + 1, dtype=dtype, scale=0.2) if bias else None
    ref = (ops_ref.f64(w) if weight else None, ops_ref.f64(b) if bias else None, kind, eps, offset)
    return binding.Norm(w, b, kind=kind, eps=eps, offset=offset), ref


def _check(r, y, after=None, before=None, gate=None, **kw):
    a = after or (None, None)
    b = before or (None, None)
    ref = ops_ref.block_norm(r, y, before=b[1], after=a[1], gate=gate,
                             **{k: v for k, v in kw.items() if k in ("gate_sigmoid", "res_scale", "out_scale")})
    got = binding.block_norm(r, y, before=b[0], after=a[0], gate=gate, **kw)
    torch.cuda.synchronize()
    ops_ref.check_norm(got[0], ref[0], ref[1])
    if before is not None:
        ops_ref.check_norm(got[1], ref[2], ref[3])
    else:
        assert got[1] is None
    return got


WIDTHS = [1, 2, 7, 8, 63, 128, 512, 513, 520, 1000, 1024, 1001, 2048, 2049, 2056, 4096, 4100, 7168, 8192, 8193, 16384,
          16400, 32768, 40000, 65535, 65536]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype,residual", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_norm_widths(H, dtype, residual):
    T = 5 if H < 20000 else 2
    print(f"block norm H={H} {dtype} {residual}", flush=True)
    r, y = _randn(T, H, seed=1, dtype=residual, scale=2.0), _randn(T, H, seed=2, dtype=dtype)
    for kind, bias, offset in (("rms", False, 1.0), ("layer", True, 0.0)):
        if kind == "layer" and H == 1:
            continue  # the difference from its own mean is 0: covered below
        _check(r, y, _make_norm(H, dtype, kind, offset, bias, 3), _make_norm(H, dtype, kind, offset, bias, 7),
               gate=_randn(H, seed=9, dtype=dtype), res_scale=0.5, out_scale=1.5)


@pytest.mark.parametrize("H", [96, 1001, 4096])
@pytest.mark.parametrize("T", [1, 4, 7, 300])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_norm_gates_and_parts(H, T, gate, sigmoid):
    print(f"block norm T={T} H={H} gate={gate} sigmoid={sigmoid}", flush=True)
    r, y = _randn(T, H, seed=1, dtype=F32), _randn(T, H, seed=2, dtype=BF16)
    g = {"none": None, "token": _randn(T, 1, seed=4, dtype=BF16), "channel": _randn(H, seed=4, dtype=BF16),
         "element": _randn(T, H, seed=4, dtype=BF16)}[gate]
    n1, n2 = _make_norm(H, BF16, "rms", 0.0, False, 5), _make_norm(H, BF16, "layer", 0.0, True, 6, eps=1e-5)
    for after, before in ((n1, n2), (None, n1), (n2, None), (None, None)):
        _check(r, y, after, before, gate=g, gate_sigmoid=sigmoid, out_scale=0.3)


def test_norm_alone_and_residual_scale():
    r = _randn(9, 256, seed=1, dtype=F16)
    n = _make_norm(256, F16, "rms", 0.0, False, 5)
    out, h = _check(r, None, None, n)
    assert out.data_ptr() == r.data_ptr()
    out, _ = _check(r, None, None, n, res_scale=0.5)
    assert out.data_ptr() != r.data_ptr()
    _check(r, None, None, _make_norm(256, F16, "layer", 0.0, False, 5, weight=False))
    r32 = _randn(9, 256, seed=1)
    h = torch.empty((9, 256), dtype=BF16, device="cuda")
    nb = _make_norm(256, BF16, "rms", 0.0, False, 5)
    _check(r32, None, None, nb, h_out=h)


def test_norm_degenerate_rows():
    """Zero rows, constant rows (no spread), one column, means far above the spread, large and tiny values."""
    H = 640
    y = _randn(7, H, seed=2, dtype=F32)
    y[0] = 0.0
    y[1] = 3.0
    y[2] += 1000.0
    y[3] *= 1e15
    y[4] *= 1e-18
    r = torch.zeros((7, H), device="cuda")
    for kind in ("rms", "layer"):
        n = _make_norm(H, F32, kind, 0.0, False, 5)
        # (rows 1 and 2 of the layer norm: the mean's binary32 error, 90 steps of its size, against a small
        # spread is part of the tolerance's term sizes)
        _check(r, y, n, None)
    one = _randn(4, 1, seed=3)
    _check(one, one.clone(), _make_norm(1, F32, "layer", 0.0, True, 5), None)


@pytest.mark.parametrize("H", [512, 515, 2048, 7168])
def test_norm_in_place_and_strides(H):
    print(f"block norm in place H={H}", flush=True)
    T = 6
    n1, n2 = _make_norm(H, BF16, "rms", 0.0, False, 5), _make_norm(H, BF16, "rms", 1.0, False, 6)
    big_r, big_y = _randn(T, H + 24, seed=1, dtype=BF16), _randn(T, H + 40, seed=2, dtype=BF16)
    for c0 in (0, 8, 3):
        r, y = big_r[:, c0:c0 + H], big_y[:, c0:c0 + H]
        g = _randn(T, H + 9, seed=4, dtype=BF16)[:, 1:H + 1]
        want = _check(r, y, n1, n2, gate=g)
        r2, y2 = big_r.clone(), big_y.clone()
        got = binding.block_norm(r2[:, c0:c0 + H], y2[:, c0:c0 + H], before=n2[0], after=n1[0], gate=g,
                                 residual_out=r2[:, c0:c0 + H], h_out=y2[:, c0:c0 + H])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for a, b in ((r2, big_r), (y2, big_y)):  # columns beside it stay as they were
            assert torch.equal(a[:, :c0], b[:, :c0]) and torch.equal(a[:, c0 + H:], b[:, c0 + H:])


def test_norm_refusals_empty_and_streams():
    r, y = _randn(4, 64, seed=1, dtype=BF16), _randn(4, 64, seed=2, dtype=BF16)
    n = binding.Norm(_randn(64, seed=3, dtype=BF16))
    got = binding.block_norm(r[:0], y[:0], before=n, after=n)
    assert got[0].shape == (0, 64) and got[1].shape == (0, 64)
    for bad in (dict(gate=_randn(65, seed=1, dtype=BF16)), dict(gate=_randn(64, seed=1)),
                dict(before=binding.Norm(_randn(64, seed=1))), dict(before=binding.Norm(_randn(63, seed=1, dtype=BF16))),
                dict(h_out=torch.empty_like(y)), dict(residual_out=torch.empty((4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            binding.block_norm(r, y, **bad)
    with pytest.raises(binding.Nvfp4Error) as e:
        binding.block_norm(r, y, before=n, h_out=r)
    assert e.value.status == "NVFP4_ERR_ALIAS"
    with pytest.raises(binding.Nvfp4Error):
        binding.block_norm(r, after=n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = binding.block_norm(r, y, before=n, after=n)
    got = binding.block_norm(r, y, before=n, after=n, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_norm_far_offsets():
    """Rows whose offsets pass 2^31 elements and 2^32 bytes."""
    ld, T, H = 1 << 23, 300, 128
    base = torch.empty((2, (T - 1) * ld + H), dtype=BF16, device="cuda")
    r, y = base[0].as_strided((T, H), (ld, 1)), base[1].as_strided((T, H), (ld, 1), (T - 1) * ld + H)
    r.copy_(_randn(T, H, seed=1))
    y.copy_(_randn(T, H, seed=2))
    n = _make_norm(H, BF16, "rms", 0.0, False, 5)
    want = _check(r, y, n, n)
    binding.block_norm(r, y, before=n[0], after=n[0], residual_out=r, h_out=y)
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])


def test_norm_graph_replay():
    r, y = _randn(33, 2048, seed=1, dtype=BF16), _randn(33, 2048, seed=2, dtype=BF16)
    n = binding.Norm(_randn(2048, seed=3, dtype=BF16))
    ro, h = torch.empty_like(r), torch.empty_like(y)
    binding.block_norm(r, y, before=n, after=n, residual_out=ro, h_out=h)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            binding.block_norm(r, y, before=n, after=n, residual_out=ro, h_out=h)
    torch.cuda.synchronize()
    for i in range(3):
        y.copy_(_randn(33, 2048, seed=30 + i))
        g.replay()
        torch.cuda.synchronize()
        want = binding.block_norm(r, y, before=n, after=n)
        assert torch.equal(ro, want[0]) and torch.equal(h, want[1])


def test_norm_rows_past_one_grid_dimension():
    """More rows than a launch has blocks in x (2^21 + 5 of 1100 columns)."""
    T, H = (1 << 21) + 5, 1100
    r = torch.zeros((T, H), dtype=BF16, device="cuda")
    r[-7:] = _randn(7, H, seed=1, dtype=BF16)
    n, ref = _make_norm(H, BF16, "rms", 0.0, False, 5)
    _, h = binding.block_norm(r, before=n)
    torch.cuda.synchronize()
    _, _, rh, hs = ops_ref.block_norm(r[-7:], None, before=ref)
    ops_ref.check_norm(h[-7:], rh, hs)
    assert not h[:-7].any()
