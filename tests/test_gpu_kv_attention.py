"""Attention over the 8-bit key-value cache against the formula in 64 bits."""
import math

import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import kv_ref

pytestmark = pytest.mark.gpu


def _run(b, heads, cu=True, window=0, scale=None, q_scale=1.0, q=None, cache=None):
    if cache is None:
        cache = b.cache(binding)
        b.append_new(binding, cache)
    q = b.queries(heads, q_scale) if q is None else q
    table, lens, slots, at = b.args()
    out = binding.kv_attention(cache, q, table, lens, slots, cu=at if cu else None, window=window, scale=scale)
    want, far = b.attention(q, scale=scale, window=window)
    kv_ref.check(out, want, far)
    return cache, q, out


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("P,kv,G", [(16, 3, 1), (32, 2, 5), (64, 1, 8), (128, 2, 16), (64, 1, 23), (16, 1, 40)])
def test_single_tokens(D, P, kv, G):
    """Every length around a page and a step of the kernel."""
    held = sorted({0, 1, P - 2, P - 1, P, 63, 64, 65, 2 * P - 1, 127, 128, 200, 511})
    b = kv_ref.Batch(held, [1] * len(held), kv, D, P, torch.bfloat16 if kv != 2 else torch.float16, seed=G)
    _run(b, kv * G, cu=False)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("P,kv,G,window", [(16, 2, 3, 0), (32, 1, 4, 100), (64, 2, 1, 0), (128, 1, 7, 33), (64, 1, 12, 1)])
def test_chunks(D, P, kv, G, window):
    """Chunks from nothing to more rows than a tile, beside single tokens, at any start."""
    held, new = [0, 37, 64, 130, 5, 200, 0, 3], [70, 1, 0, 150, 2, 33, 1, 300]
    b = kv_ref.Batch(held, new, kv, D, P, torch.float16 if G % 2 else torch.bfloat16, seed=P)
    _run(b, kv * G, window=window)


@pytest.mark.parametrize("D,G", [(128, 4), (256, 2), (64, 1)])
def test_one_sequence(D, G):
    for held, new in ((0, 1), (0, 5), (100, 20), (0, 400), (129, 260)):
        b = kv_ref.Batch([held], [new], 2, D, 64, seed=new)
        _run(b, 2 * G)


@pytest.mark.parametrize("D,P,G,dtype", [(128, 64, 8, torch.bfloat16), (64, 16, 4, torch.float16),
                                         (256, 128, 3, torch.bfloat16), (192, 32, 20, torch.float16)])
def test_long_sequences_in_pieces(D, P, G, dtype):
    held = [5000, 1, 2047, 130, 0, 777]
    b = kv_ref.Batch(held, [1] * 6, 2, D, P, dtype)
    cache, q, out = _run(b, 2 * G, cu=False)
    table, lens, slots, cu = b.args()
    for _ in range(3):  # the same bits again, with and without cu
        again = binding.kv_attention(cache, q, table, lens, slots)
        assert torch.equal(out, again)
    _run(b, 2 * G, q=q, cache=cache)
    _run(b, 2 * G, q=q, cache=cache, window=900, cu=False)


@pytest.mark.parametrize("D,P,G", [(128, 64, 4), (64, 16, 3), (256, 64, 2), (192, 128, 1)])
def test_long_chunks_in_pieces(D, P, G):
    b = kv_ref.Batch([3000, 1200, 2500, 10], [100, 300, 1, 65], 2, D, P)
    _run(b, 2 * G)
    b = kv_ref.Batch([3000], [100], 1, D, P)
    _run(b, G)
    _run(b, G, window=1500)


def test_peaked_and_flat_scores():
    b = kv_ref.Batch([700, 90], [40, 1], 2, 128, 64)
    cache, q, _ = _run(b, 8, q_scale=12.0)
    _run(b, 8, q=q, cache=cache, scale=0.0)
    _run(b, 8, q=q, cache=cache, scale=-0.02)
    _run(b, 8, q_scale=1e-3, cache=cache)


def test_subnormal_fp16_queries():
    """Products with numbers below fp16's normal range are not dropped."""
    b = kv_ref.Batch([150], [4], 1, 64, 64, torch.float16)
    q = (b.queries(2).float() * 2.0 ** -18).to(torch.float16)
    _run(b, 2, q=q, scale=2.0 ** 15)
    b = kv_ref.Batch([150], [40], 1, 128, 16, torch.float16)
    q = (b.queries(2).float() * 2.0 ** -18).to(torch.float16)
    _run(b, 2, q=q, scale=-(2.0 ** 15))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_growing_scores_and_values(dtype):
    """The running maximum and the values' unit grow with nearly every page."""
    P, n = 16, 800
    b = kv_ref.Batch([n], [2], 1, 64, P, dtype)
    grow = torch.exp2(torch.arange(n + 2, dtype=torch.float32) / 100)[:, None, None]
    b.k_all[0] = (b.k_all[0].float().abs() * grow / 16).to(dtype)
    b.v_all[0] = (b.v_all[0].float() * grow).to(dtype)
    q = torch.ones((2, 4, 64), dtype=dtype, device="cuda")
    _run(b, 4, q=q)
    b.k_all[0], b.v_all[0] = b.k_all[0].flip(0), b.v_all[0].flip(0)
    _run(b, 4, q=q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_of_very_different_size(dtype):
    """A page of huge values out of reach of the softmax, pages of zeros, tiny values."""
    P = 32
    b = kv_ref.Batch([200], [3], 2, 64, P, dtype)
    for x in (b.v_all[0],):
        x[0:P] = (x[0:P].float() * 1000).to(dtype)
        x[P:2 * P] = 0.0
        x[2 * P:] = (x[2 * P:].float() * 1e-3).to(dtype)
    b.k_all[0][0:P] = (-b.k_all[0][0:P].float().abs() * 20).to(dtype)
    q = torch.rand((3, 4, 64), generator=b.gen).to(dtype).cuda()
    _run(b, 4, q=q)
    b.v_all[0][:] = 0.0
    _run(b, 4, q=q)


def test_queries_far_below_and_above_one():
    b = kv_ref.Batch([150], [4], 1, 128, 64)
    q = b.queries(2)
    q[0] *= 2.0 ** -60
    q[1] *= 2.0 ** -7
    q[3, 0] = 0.0
    _run(b, 2, q=q)
    b = kv_ref.Batch([150], [4], 1, 128, 64, scale=2.0 ** -40)
    q = (b.queries(2).float() * 2.0 ** 40).to(torch.bfloat16)
    _run(b, 2, q=q)


def test_nan_stays_with_those_who_see_it():
    """A NaN page, a NaN token in the tail, a NaN query."""
    P = 16
    for which in ("k", "v"):
        for at in (20, 203, 209):  # in an old page, in one that the call completes, in the tail
            b = kv_ref.Batch([190], [20], 2, 64, P)
            getattr(b, which + "_all")[0][at, 1, 3] = float("nan")
            cache, q, out = _run(b, 6)
            assert torch.isnan(out).any() and not torch.isnan(out[:, :3]).any()
            _run(b, 6, q=q, cache=cache, window=100)
    b = kv_ref.Batch([100], [40], 1, 64, P)
    q = b.queries(3)
    q[7, 1, 5] = float("nan")
    q[9, 2, 5] = float("inf")
    cache = b.cache(binding)
    b.append_new(binding, cache)
    table, lens, slots, cu = b.args()
    out = binding.kv_attention(cache, q, table, lens, slots, cu=cu)
    bad = torch.isnan(out).any(2).nonzero().tolist()
    assert bad == [[7, 1], [9, 2]]
    clean = q.clone()
    clean[7, 1], clean[9, 2] = 0.0, 0.0
    want, far = b.attention(clean)
    out[7, 1], out[9, 2] = 0.0, 0.0
    want[7, 1], want[9, 2] = 0.0, 0.0
    kv_ref.check(out, want, far)


@pytest.mark.parametrize("new", [1, 60])
def test_pages_outside_the_cache_hold_nothing(new):
    """Some pages missing, and a sequence without any: rows that see no key are zero."""
    P = 16
    b = kv_ref.Batch([160, 15 if new == 1 else 32], [new, new], 2, 64, P)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(4)
    table, lens, slots, cu = b.args()
    table[0, 2], table[0, 5] = -1, b.pages
    total = [160 + new, b.held[1] + new]
    table[1] = -5
    hidden = [torch.zeros(total[0], dtype=torch.bool), torch.zeros(total[1], dtype=torch.bool)]
    hidden[0][2 * P:3 * P] = hidden[0][5 * P:6 * P] = True
    hidden[1][:total[1] // P * P] = True
    out = binding.kv_attention(cache, q, table, lens, slots, cu=cu)
    want, far = b.attention(q, hidden=hidden)
    kv_ref.check(out, want, far)
    if new == 1:
        assert (out[1] == 0).all()  # its only page was completed by this token


def test_padding_and_rows_behind_the_last_sequence_stay():
    b = kv_ref.Batch([40, 3, 2000], [1, 1, 1], 2, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(6)
    table, lens, slots, cu = b.args()
    want, far = b.attention(q)
    for lens_, slots_ in ((b.ints([40, -1, 2000]), slots), (lens, b.ints([slots[0], -1, slots[2]])),
                          (b.ints([40, 10 ** 8, 2000]), slots), (lens, b.ints([slots[0], 77, slots[2]]))):
        for at in (None, cu):
            out = torch.full_like(q, 5.0)
            binding.kv_attention(cache, q, table, lens_, slots_, cu=at, out=out)
            assert (out[1] == 5.0).all()
            kv_ref.check(out[::2], want[::2], far[::2])
    more = torch.cat((q, q))
    out = torch.full_like(more, 5.0)
    binding.kv_attention(cache, more, table, lens, slots, cu=cu, out=out)
    assert (out[3:] == 5.0).all()
    kv_ref.check(out[:3], want, far)


def test_entries_that_share_tokens_harm_nothing():
    b = kv_ref.Batch([2000] * 8, [64] * 8, 1, 64, 16)
    cache = b.cache(binding)
    q = torch.randn((64, 8, 64), device="cuda", dtype=torch.bfloat16)
    table, lens, slots, _ = b.args()
    for cu in ([0, 64, 0, 64, 0, 64, 0, 64, 0], [64, 0, 64, 0, 64, 0, 64, 0, 64], [0, 10 ** 9, 0, 3, -1, 5, 2, 1, 0]):
        binding.kv_attention(cache, q, table, lens, slots, cu=b.ints(cu))
    torch.cuda.synchronize()


def test_strided_queries_and_outputs():
    b = kv_ref.Batch([100, 7], [30, 1], 2, 128, 32)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(6)
    want, far = b.attention(q)
    table, lens, slots, cu = b.args()
    wide = torch.full((31, 10, 128 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8, :128] = q
    to = torch.full((8, 31, 128 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = to[1:7, :, :128].transpose(0, 1)
    got = binding.kv_attention(cache, wide[:, 2:8, :128], table, lens, slots, cu=cu, out=out)
    assert got is out or got.data_ptr() == out.data_ptr()
    kv_ref.check(out, want, far)
    assert (to[0] == 3.0).all() and (to[7] == 3.0).all() and (to[:, :, 128:] == 3.0).all()
    # a table whose rows are further apart, and wider than the call's
    big = torch.full((2, 50), -9, dtype=torch.int32, device="cuda")
    big[:, 3:3 + table.shape[1]] = table
    got = binding.kv_attention(cache, q, big[:, 3:3 + table.shape[1]], lens, slots, cu=cu)
    kv_ref.check(got, want, far)


@pytest.mark.parametrize("D,G,new", [(128, 8, 8), (64, 8, 5), (192, 8, 5), (256, 3, 9), (128, 1, 97), (64, 4, 12), (128, 3, 17)])
def test_entries_of_a_few_tokens(D, G, new):
    """Between single tokens and chunks: entries of one to four tiles of the kernel for few rows, alike and mixed
    with others, short and cut into pieces."""
    b = kv_ref.Batch([1500, 0, 77, 300], [new] * 4, 2, D, 32)
    _run(b, 2 * G)
    b = kv_ref.Batch([1500, 64, 3, 0, 10], [new, 1, 200, new, 0], 1, D, 64, torch.float16)
    _run(b, G)
    _run(b, G, window=70)


def test_no_tokens():
    b = kv_ref.Batch([20], [1], 2, 64, 16)
    cache = b.cache(binding)
    table, lens, slots, _ = b.args()
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert binding.kv_attention(cache, q, table, lens, slots, cu=b.ints([0, 0])).shape == (0, 4, 64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert binding.kv_attention(cache, q, table[:0], none, none).shape == (0, 4, 64)


def test_many_entries():
    """More entries than a block has threads, most of them short."""
    held = [(i * 37) % 90 for i in range(700)]
    b = kv_ref.Batch(held, [1] * 700, 1, 64, 16)
    _run(b, 2, cu=False)
    b = kv_ref.Batch(held, [i % 3 for i in range(700)], 1, 64, 16)
    _run(b, 2)
    held[333] = 4000
    b = kv_ref.Batch(held, [1] * 700, 1, 64, 16)
    _run(b, 2, cu=False)


def test_scale_default():
    b = kv_ref.Batch([30], [1], 1, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(2)
    table, lens, slots, _ = b.args()
    assert torch.equal(binding.kv_attention(cache, q, table, lens, slots),
                       binding.kv_attention(cache, q, table, lens, slots, scale=1 / math.sqrt(64)))
