"""Routing by scores, bias and groups on the GPU against the 64-bit rule: ids
exactly, weights within the rounding to binary32."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import ops_ref

pytestmark = pytest.mark.gpu

# A renormalized or sigmoid weight is formed in binary64 and rounded once (half a step, 2^-24); without
# renormalization the softmax sum is of binary32 exponentials: each within 2 steps, its argument's rounding
# at most the mean distance from the largest logit, below ln 1024 = 7 steps, in relative terms.
TOL_ROUNDED, TOL_SUM = 1.01 * 2.0 ** -24, 10.5 * 2.0 ** -24


def _check(logits, k, bias=None, out=None, stream=None, **rule):
    ids, w = binding.route(logits, k, binding.Router(**rule), bias=bias, out=out, stream=stream)
    torch.cuda.synchronize()
    rids, rw = ops_ref.route(logits, k, bias=bias, **rule)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    tol = TOL_SUM if rule.get("score", "softmax") == "softmax" and not rule.get("renormalize", True) else TOL_ROUNDED
    # (a weight below the smallest normal binary32 has an absolute half step of 2^-150)
    np.testing.assert_allclose(w.double().cpu().numpy(), rw, rtol=tol, atol=2.0 ** -150)
    return ids, w


def _logits(T, E, seed=0, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, E), generator=g) + 0.5 * torch.randn(E, generator=g)).to(dtype).cuda()


def _bias(E, seed=0):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed + 99))).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", [
    (1, 1, 1, 1, 1, 1), (3, 8, 8, 1, 1, 1), (5, 16, 4, 4, 2, 2), (1, 128, 8, 1, 1, 1), (64, 256, 8, 8, 4, 2),
    (33, 60, 4, 5, 2, 1), (9, 300, 16, 6, 3, 2), (7, 1024, 16, 64, 9, 2), (2, 1000, 16, 1, 1, 1), (4, 64, 2, 64, 3, 2),
    (1025, 16, 2, 1, 1, 1), (1030, 20, 3, 4, 2, 2), (1100, 64, 6, 8, 3, 1), (1500, 100, 9, 50, 12, 2),
    (2000, 256, 8, 8, 4, 2), (1201, 256, 16, 64, 5, 1), (1027, 300, 16, 6, 3, 1),
    (2100, 160, 8, 8, 4, 2), (2049, 150, 5, 3, 2, 1), (2065, 192, 16, 8, 4, 2), (2100, 300, 16, 6, 3, 2), (2061, 320, 8, 4, 2, 2), (2050, 384, 8, 6, 3, 2), (2077, 384, 5, 8, 4, 1),
    (2049, 432, 16, 3, 2, 2), (2055, 433, 7, 1, 1, 1), (2060, 510, 9, 6, 3, 2), (2052, 1000, 16, 5, 3, 2)])
def test_route_sizes(T, E, k, groups, top_groups, best, score, bias):
    print(f"route T={T} E={E} k={k} groups={groups}/{top_groups}/{best} {score} bias={bias}", flush=True)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        _check(_logits(T, E), k, _bias(E) if bias else None, score=score, groups=groups, top_groups=top_groups,
               group_best=best, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [40, 1200])
def test_route_16_bit_ties_and_strides(dtype, T):
    """16-bit logits tie; ties go to the lower expert; rows further apart than E."""
    print(f"route {dtype} T={T}", flush=True)
    base = _logits(T, 96, dtype=dtype)
    base[:, 3] = base[:, 70]
    base[1] = 0.0
    base[2, ::2] = -0.0
    base[2, 1::2] = 0.0
    for view in (base, base[:, 16:80], base[::2, :64]):
        for rule in (dict(), dict(groups=8, top_groups=3, group_best=2), dict(score="sigmoid", groups=4, top_groups=2)):
            _check(view, 7, **rule)
            _check(view, 7, bias=torch.zeros(view.shape[1], device="cuda"), **rule)


@pytest.mark.parametrize("T,E", [(12, 64), (1100, 64), (12, 512)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masks(T, E, score, bias):
    """Masked logits and biases, rows with fewer open experts than k or none, NaN and infinities, far logits."""
    print(f"route masks T={T} E={E} {score} bias={bias}", flush=True)
    l = _logits(T, E, 3)
    low = torch.finfo(torch.float32).min
    inf = float("inf")
    l[0] = -inf
    l[1] = float("nan")
    l[2] = -inf
    l[2, E - 1] = 0.25
    l[3] = low
    l[4, ::3] = -inf
    l[5, 5] = inf
    l[6, 7], l[6, 9] = inf, inf
    l[7, : E // 2] = -inf
    l[8] = -300.0
    l[8, 11] = 300.0
    l[9, 4] = float("nan")
    l[10] = 60.0 + 0.01 * torch.arange(E, device="cuda")
    l[11] = -2000.0 - torch.arange(E, device="cuda")
    b = _bias(E) if bias else None
    if bias:
        b[2], b[E - 2], b[6] = -inf, float("nan"), 3.0
    for rule in (dict(), dict(renormalize=False), dict(groups=8, top_groups=2, group_best=2),
                 dict(groups=4, top_groups=2)):
        _check(l, 6, b, score=score, **rule)


def test_route_close_values_keep_their_order():
    """Values nearer than binary32 can tell apart: sigmoid scores plus a bias near 1000."""
    g = torch.Generator().manual_seed(5)
    l = (0.001 * torch.randn((1100, 128), generator=g)).cuda()
    b = torch.full((128,), 1000.0).cuda()
    _check(l, 8, b, score="sigmoid")
    _check(l[:50], 8, b, score="softmax", groups=8, top_groups=4, group_best=2)


def test_route_chosen_far_below_the_largest():
    """A bias that prefers experts whose softmax scores are tiny: their renormalized weights stay exact."""
    l = _logits(20, 32, 7)
    l[:, 0] = 150.0
    b = torch.zeros(32).cuda()
    b[8:16] = 5.0
    _check(l, 4, b)


def test_route_empty_and_outputs():
    ids, w = binding.route(torch.empty((0, 16), device="cuda"), 4, binding.Router())
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    out = (torch.full((6, 3), -7, dtype=torch.int32, device="cuda"), torch.full((6, 3), -7.0, device="cuda"))
    l = _logits(4, 16)
    _check(l, 3, out=(out[0][1:5], out[1][1:5]))
    for o in out:  # rows beside the batch stay as they were
        assert (o[0] == -7).all() and (o[5] == -7).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _check(l, 3, stream=s)
    _check(l, 3, group_best=2)  # without groups it has no effect
    for bad in (dict(groups=3), dict(groups=4, top_groups=1, group_best=2)):
        with pytest.raises(binding.Nvfp4Error):
            binding.route(l, 8, binding.Router(**bad))
    with pytest.raises(ValueError):
        binding.route(l, 2, binding.Router(), bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        binding.route(l.t(), 2, binding.Router())
    with pytest.raises(TypeError):
        binding.route(l, 2, binding.Norm())
    with pytest.raises(TypeError):
        binding.block_norm(l, before=binding.Router())
    for k in (0, -1, 17, 1 << 40):
        with pytest.raises(binding.Nvfp4Error) as e:
            binding.route(l, k, binding.Router())
        assert e.value.status == "NVFP4_ERR_INVALID_ARG"


def test_route_far_offsets():
    """Rows whose offsets pass 2^31 elements and 2^32 bytes."""
    ld, T = 1 << 23, 300
    base = torch.empty(((T - 1) * ld + 64,), dtype=torch.bfloat16, device="cuda")
    l = base.as_strided((T, 64), (ld, 1))
    l.copy_(_logits(T, 64))
    _check(l, 6, groups=8, top_groups=4, group_best=2)


@pytest.mark.parametrize("T", [3, 1500])
def test_route_graph_replay(T):
    l, b = _logits(T, 256), _bias(256)
    r = binding.Router(score="sigmoid", groups=8, top_groups=4, group_best=2, scale=2.5)
    out = (torch.empty((T, 8), dtype=torch.int32, device="cuda"), torch.empty((T, 8), device="cuda"))
    binding.route(l, 8, r, bias=b, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            binding.route(l, 8, r, bias=b, out=out)
    torch.cuda.synchronize()
    for i in range(3):
        l.copy_(_logits(T, 256, seed=20 + i))
        g.replay()
        torch.cuda.synchronize()
        ids, w = binding.route(l, 8, r, bias=b)
        assert torch.equal(ids, out[0]) and torch.equal(w, out[1])


def test_route_tokens_past_one_grid_dimension():
    """More tokens than a launch has blocks in x of 16 tokens each (2^25 + 21)."""
    T = (1 << 25) + 21
    l = torch.zeros((T, 4), dtype=torch.bfloat16, device="cuda")
    l[-30:] = _logits(30, 4, dtype=torch.bfloat16)
    ids, w = binding.route(l, 2, binding.Router())
    torch.cuda.synchronize()
    rids, rw = ops_ref.route(l[-30:], 2)
    np.testing.assert_array_equal(ids[-30:].cpu().numpy(), rids)
    np.testing.assert_allclose(w[-30:].double().cpu().numpy(), rw, rtol=TOL_ROUNDED)
    assert (w[:-30] == 0.5).all() and (ids[:-30, 1] == 1).all()
