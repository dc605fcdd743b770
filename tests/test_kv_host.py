"""Argument checks of the key-value cache's operators (no GPU needed): each refusal returns its documented
status before any device work; empty calls are no-ops; the references of the GPU tests pinned on the CPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import kv_ref

P = ctypes.c_void_p
BF16, F16, F32 = 0, 1, 2
MB = 1 << 20


def _cache(**kw):
    c = dict(num_pages=10, num_slots=4, kv_heads=2, head_dim=64, page_size=16, codes=1 * MB, scales=2 * MB, tails=3 * MB,
             tail_scales=4 * MB)
    c.update(kw)
    return binding.KvCacheDesc(*c.values())


def _batch(**kw):
    b = dict(entries=3, tokens=3, table=5 * MB, table_width=5, ld_table=5, lens=6 * MB, slots=7 * MB, cu=0)
    b.update(kw)
    return binding.KvBatchDesc(*b.values())


def _append(c=None, b=None, k=8 * MB, ld_k=128, lh_k=64, v=9 * MB, ld_v=128, lh_v=64, dtype=BF16):
    return binding.lib().kv_append(c or _cache(), b or _batch(), P(k), ld_k, lh_k, P(v), ld_v, lh_v, dtype, None)


def _attention(c=None, b=None, q=8 * MB, ld_q=256, lh_q=64, heads=4, dtype=BF16, scale=0.1, window=0, ws=10 * MB, nws=0,
               out=9 * MB, ld_o=256, lh_o=64):
    return binding.lib().kv_attention(c or _cache(), b or _batch(), P(q), ld_q, lh_q, heads, dtype, scale, window, P(ws),
                                      nws, P(out), ld_o, lh_o, None)


def _read(c=None, b=None, k=8 * MB, v=9 * MB, dtype=F32):
    return binding.lib().kv_read(c or _cache(), b or _batch(), P(k), P(v), dtype, None)


def _fork(c=None, b=None, src=8 * MB, dst=9 * MB, pairs=2):
    return binding.lib().kv_fork(c or _cache(), b or _batch(), P(src), P(dst), pairs, None)


CALLS = (_append, _attention, _read, _fork)


@pytest.mark.parametrize("call", CALLS)
def test_sizes_and_pointers(call):
    for bad in (dict(num_pages=0), dict(num_pages=2 ** 31), dict(num_slots=0), dict(num_slots=2 ** 31), dict(kv_heads=0),
                dict(kv_heads=1025), dict(head_dim=32), dict(head_dim=96), dict(head_dim=320), dict(head_dim=0),
                dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(page_size=0), dict(codes=0),
                dict(scales=0), dict(tails=0), dict(tail_scales=0), dict(codes=MB + 8), dict(scales=2 * MB + 4),
                dict(tails=3 * MB + 2), dict(tail_scales=4 * MB + 4)):
        assert call(c=_cache(**bad)) == 1, bad
    for bad in (dict(entries=-1), dict(entries=2 ** 31 - 1), dict(table_width=0), dict(table_width=2 ** 26 + 1, ld_table=2 ** 27),
                dict(ld_table=4), dict(ld_table=2 ** 31 + 1), dict(table=0), dict(lens=0), dict(slots=0), dict(table=5 * MB + 2),
                dict(lens=6 * MB + 1), dict(slots=7 * MB + 2)):
        assert call(b=_batch(**bad)) == 1, bad
    if call is not _fork:
        for bad in (dict(tokens=-1), dict(tokens=2 ** 31), dict(tokens=4), dict(cu=6 * MB + 6)):
            assert call(b=_batch(**bad)) == 1, bad
    L = binding.lib()
    assert L.kv_append(None, _batch(), P(MB), 128, 64, P(MB), 128, 64, BF16, None) == 1
    assert L.kv_read(_cache(), None, P(MB), P(MB), F32, None) == 1
    assert L.kv_fork(None, None, P(MB), P(MB), 1, None) == 1


def test_append_refusals():
    assert _append(dtype=F32) == 1 and _append(dtype=7) == 1
    assert _append(k=0) == 1 and _append(v=0) == 1 and _append(k=8 * MB + 8) == 1 and _append(v=9 * MB + 2) == 1
    for bad in (dict(ld_k=129), dict(ld_v=4), dict(lh_k=-8), dict(lh_v=2 ** 31 + 8), dict(ld_k=-128)):
        assert _append(**bad) == 1, bad
    assert _append(k=1 * MB + 64) == 3 and _append(v=2 * MB) == 3 and _append(k=3 * MB + 16) == 3 and _append(v=4 * MB) == 3
    assert _append(b=_batch(table=1 * MB)) == 3 and _append(b=_batch(lens=3 * MB)) == 3
    assert _append(b=_batch(entries=1 << 30, tokens=1 << 30), c=_cache(kv_heads=64)) == 1  # more blocks than a launch has
    assert _append(b=_batch(entries=0, tokens=0, table=0, lens=0, slots=0), k=0, v=0) == 0
    assert _append(b=_batch(tokens=0, cu=6 * MB), k=0, v=0) == 0


def test_attention_refusals():
    assert _attention(dtype=F32) == 1 and _attention(heads=0) == 1 and _attention(heads=3) == 1
    assert _attention(heads=130, ld_q=130 * 64, ld_o=130 * 64) == 1  # 65 a kv head
    for bad in (dict(scale=math.inf), dict(scale=math.nan), dict(window=-1), dict(q=0), dict(out=0), dict(q=8 * MB + 2),
                dict(out=9 * MB + 8), dict(ld_q=100), dict(lh_o=63), dict(ld_o=192), dict(lh_o=56), dict(ld_o=0), dict(lh_o=0)):
        assert _attention(**bad) == 1, bad
    # heads before tokens is an order, too (checked as far as the overlap with the cache)
    assert _attention(ld_o=64, lh_o=64 * 2) == 1 and _attention(ld_o=64, lh_o=64 * 3, out=1 * MB) == 3
    assert _attention(out=8 * MB + 512) == 3 and _attention(out=2 * MB) == 3 and _attention(out=4 * MB - 16) == 3
    assert _attention(b=_batch(slots=9 * MB + 4)) == 3
    long = _batch(table_width=100, ld_table=100)
    need = ctypes.c_int64()
    assert binding.lib().kv_attention_workspace(_cache(), long, 4, ctypes.byref(need)) == 0 and need.value > 0
    assert _attention(b=long, ws=0, nws=need.value) == 1 and _attention(b=long, nws=need.value - 1) == 1
    assert _attention(b=long, ws=10 * MB + 8, nws=need.value) == 1 and _attention(b=long, ws=8 * MB, nws=need.value) == 3
    assert _attention(b=_batch(tokens=2 ** 29, cu=6 * MB)) == 1  # too many rows
    assert _attention(b=_batch(entries=0, tokens=0, table=0), q=0, out=0, ws=0) == 0


def test_workspace():
    def need(heads=4, c=None, **b):
        n = ctypes.c_int64(-1)
        status = binding.lib().kv_attention_workspace(c or _cache(), _batch(**b), heads, ctypes.byref(n))
        return (status, n.value)
    assert need() == (0, 0) and need(entries=0, tokens=0) == (0, 0)      # short tables are never cut
    assert need(heads=5)[0] == 1 and need(tokens=-1)[0] == 1
    assert binding.lib().kv_attention_workspace(_cache(), _batch(), 4, None) == 1
    wide = dict(table_width=1 << 12, ld_table=1 << 12)
    one, many = need(**wide)[1], need(entries=4096, tokens=4096, **wide)[1]
    assert 0 < one <= many < 1 << 28
    assert 0 < need(entries=4096, tokens=10 ** 6, cu=6 * MB, **wide)[1] < 1 << 29


def test_read_and_fork_refusals():
    assert _read(dtype=3) == 1 and _read(k=0) == 1 and _read(v=0) == 1 and _read(k=8 * MB + 4) == 1
    assert _read(k=1 * MB) == 3 and _read(v=8 * MB + 256) == 3 and _read(v=3 * MB + 16) == 3
    assert _read(b=_batch(lens=8 * MB)) == 3
    assert _read(b=_batch(entries=0, tokens=0, table=0), k=0, v=0) == 0
    assert _fork(pairs=-1) == 1 and _fork(pairs=2 ** 31) == 1 and _fork(src=0) == 1 and _fork(dst=0) == 1
    assert _fork(src=8 * MB + 2) == 1 and _fork(dst=6 * MB) == 3 and _fork(src=5 * MB + 8) == 3
    assert _fork(b=_batch(table=3 * MB)) == 3 and _fork(b=_batch(table=6 * MB)) == 3
    assert _fork(pairs=1 << 30) == 1
    assert _fork(pairs=0, src=0, dst=0) == 0 and _fork(b=_batch(entries=0, table=0, lens=0, slots=0)) == 0


def test_cache_refusals():
    for bad in ((0, 1, 1, 64), (1, 0, 1, 64), (1, 1, 0, 64), (1, 1, 1025, 64), (1, 1, 1, 80), (2 ** 31, 1, 1, 64)):
        with pytest.raises(ValueError):
            binding.KvCache(*bad, device="cpu")
    with pytest.raises(ValueError):
        binding.KvCache(1, 1, 1, 64, page_size=24, device="cpu")


def test_reference_page():
    """A page by hand: scale 2 / 127, one tie that goes to the even code, zeros, a NaN."""
    x = np.zeros((16, 64))
    x[0, 0], x[1, 1], x[2, 2] = 2.0, -1.0, 2.0 / 127 * 0.5
    y = kv_ref.page_values(x)
    scale = np.float32(2.0) / np.float32(127.0)
    assert y[0, 0] == np.float32(127) * scale and y[1, 1] in (np.float32(-63) * scale, np.float32(-64) * scale)
    assert abs(y[2, 2]) <= scale and y[3, 3] == 0
    assert (kv_ref.page_values(np.full((16, 64), 2.0 ** -120)) == 0).all()
    x[5, 5] = np.inf
    assert np.isnan(kv_ref.page_values(x)).all()


def test_reference_attention():
    """Against torch's softmax in 64 bits, and by its own definition: equal keys give the mean of the values."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 4, 64), (10, 2, 64), (10, 2, 64)))
    out, far = kv_ref.attention(q, k, v, 7, 0.125)
    for t in range(3):
        for h in range(4):
            w = torch.softmax(0.125 * k[:8 + t, h // 2] @ q[t, h], 0)
            assert torch.allclose(out[t, h], w @ v[:8 + t, h // 2], atol=1e-13)
    assert (far > 0).all()
    out, _ = kv_ref.attention(q, torch.ones_like(k), v, 7, 0.125, window=3)
    assert torch.allclose(out[0, 0], v[5:8, 0].mean(0), atol=1e-13)
    out, _ = kv_ref.attention(q, k, v, 7, 0.125, hidden=torch.ones(10, dtype=torch.bool))
    assert (out == 0).all()
