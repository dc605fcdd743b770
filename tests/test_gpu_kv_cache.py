"""The key-value cache: what it holds after appends of every kind, read back, against
the quantization's definition, bit for bit; sequences that continue others."""
import numpy as np
import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import kv_ref

pytestmark = pytest.mark.gpu


def _read(b, cache, first, count, dtype=torch.float32):
    table, lens, slots, cu = b.args(first, count)
    return binding.kv_read(cache, table, lens, slots, cu=cu, tokens=sum(count), dtype=dtype)


def _check_all(b, cache, total, dtype=torch.float32):
    """All tokens of sequences with `total` tokens each, as the cache should hold them."""
    k, v = _read(b, cache, [0] * len(total), total, dtype)
    for got, raw in ((k, b.k_all), (v, b.v_all)):
        want = torch.cat([kv_ref.held_values(x[:n], b.P) for x, n in zip(raw, total)]).to(dtype)
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(got.cpu().nan_to_num(), want.nan_to_num())


SIZES = [(D, P, kv) for D in (64, 128, 192, 256) for P, kv in ((16, 3), (32, 1), (64, 2), (128, 5))]


@pytest.mark.parametrize("D,P,kv", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompts_of_every_length(D, P, kv, dtype):
    total = [1, P - 1, P, P + 1, 0, 2 * P, 3 * P - 5, 2]
    b = kv_ref.Batch([0] * 8, total, kv, D, P, dtype, seed=D + P)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    _check_all(b, cache, total)
    _check_all(b, cache, total, dtype)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (192, 32), (256, 128)])
def test_the_same_whatever_the_split(D, P):
    """One call, single tokens and ragged chunks leave the same cache."""
    total = [2 * P + 3, P, 3 * P - 1, 5]
    b = kv_ref.Batch([0] * 4, total, 2, D, P, seed=1)
    rng = np.random.default_rng(P)
    caches = []
    for way in ("once", "tokens", "chunks"):
        cache = b.cache(binding)
        have = [0] * 4
        while have != total:
            left = [t - h for t, h in zip(total, have)]
            if way == "once":
                n = left
            elif way == "tokens":
                n = [min(1, x) for x in left]
            else:
                n = [int(rng.integers(0, min(x, P + 9) + 1)) for x in left]
            table, lens, slots, cu = b.args(have, n)
            k, v = b.cut(b.k_all, have, n), b.cut(b.v_all, have, n)
            if n == [1] * 4:
                binding.kv_append(cache, k, v, table, lens, slots)
            else:
                binding.kv_append(cache, k, v, table, lens, slots, cu=cu)
            have = [h + x for h, x in zip(have, n)]
        _check_all(b, cache, total)
        caches.append(cache)
    for c in caches[1:]:
        used = b.table_cpu[b.table_cpu >= 0].long()
        full = torch.cat([b.table_cpu[i, :t // P] for i, t in enumerate(total)]).long().cuda()
        assert torch.equal(c.codes[full], caches[0].codes[full]) and torch.equal(c.scales[full], caches[0].scales[full])
        assert used.numel() > 0


def test_strided_keys_and_values_out_of_one_projection():
    b = kv_ref.Batch([0, 5], [70, 40], 2, 128, 32)
    cache = b.cache(binding)
    k, v = b.cut(b.k_all, b.held, b.new), b.cut(b.v_all, b.held, b.new)
    qkv = torch.full((110, 9 * 128 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, 512:768] = k.view(110, 256)
    qkv[:, 768:1024] = v.view(110, 256)
    heads = qkv[:, :1152].view(110, 9, 128)
    table, lens, slots, cu = b.args()
    binding.kv_append(cache, heads[:, 4:6], heads[:, 6:8], table, lens, slots, cu=cu)
    _check_all(b, cache, [70, 45])


def test_heads_before_tokens():
    b = kv_ref.Batch([3], [50], 3, 64, 16)
    cache = b.cache(binding)
    k, v = (b.cut(x, b.held, b.new).transpose(0, 1).contiguous().transpose(0, 1) for x in (b.k_all, b.v_all))
    table, lens, slots, cu = b.args()
    binding.kv_append(cache, k, v, table, lens, slots, cu=cu)
    _check_all(b, cache, [53])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_at_the_ends_of_the_range(dtype):
    """Zeros, infinities, NaN, the largest and the smallest numbers, in full pages and in the tail."""
    P, D = 16, 64
    total = 7 * P + 9
    b = kv_ref.Batch([0], [total], 2, D, P, dtype)
    f = torch.finfo(dtype)
    for x in (b.k_all[0], b.v_all[0]):
        x[0:P] = 0.0
        x[P + 3, 0, 5] = float("inf")
        x[2 * P + 1, 1, 7] = float("nan")
        x[3 * P:4 * P] = f.smallest_normal / 2
        x[4 * P, :, 0] = f.max
        x[5 * P:6 * P, 0] = f.tiny if dtype == torch.float16 else 2.0 ** -120
        t = 7 * P
        x[t] = 0.0
        x[t + 1, 0, 3] = float("-inf")
        x[t + 2, 1, 4] = float("nan")
        x[t + 3] = f.max
        x[t + 4] = f.smallest_normal / 2
        x[t + 5] = -f.smallest_normal
        x[t + 6] = 1.0
        x[t + 6, :, 1::2] = 2.0 ** -12
    cache = b.cache(binding)
    b.append_new(binding, cache)
    _check_all(b, cache, [total])


def test_quantized_from_the_values_as_they_came():
    """A page whose first tokens waited in the tail has the codes of one appended whole, whatever their spread."""
    P, D = 32, 128
    b = kv_ref.Batch([0, 0], [P, P], 1, D, P)
    x = b.k_all[0] * torch.exp2(torch.arange(P, dtype=torch.float32) / 2 - 8)[:, None, None].to(torch.bfloat16)
    b.k_all[0], b.k_all[1], b.v_all[0], b.v_all[1] = x, x.clone(), x.clone(), x.clone()
    cache = b.cache(binding)
    for have, n in (([0, 0], [P, 7]), ([P, 7], [0, 24]), ([P, 31], [0, 1])):
        table, lens, slots, cu = b.args(have, n)
        binding.kv_append(cache, b.cut(b.k_all, have, n), b.cut(b.v_all, have, n), table, lens, slots, cu=cu)
    _check_all(b, cache, [P, P])


def test_numbers_near_ties_are_rounded_as_defined():
    P, D = 64, 128
    b = kv_ref.Batch([0], [P], 1, D, P, torch.float16)
    x = torch.arange(P * D, dtype=torch.float32).reshape(P, 1, D) % 509 - 254
    x[0, 0, 0] = 254.0
    b.k_all[0] = x.to(torch.float16)
    b.v_all[0] = (x * 0.37).to(torch.float16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    _check_all(b, cache, [P])


@pytest.mark.parametrize("back", [32 + 3, 32, 16])
def test_tokens_taken_back(back):
    """To inside the incomplete page, to its start, to the end of an older page; other tokens come instead."""
    P, D = 16, 64
    b = kv_ref.Batch([45], [30], 2, D, P)
    cache = b.cache(binding)
    for x in (b.k_all, b.v_all):
        x[0] = torch.cat((x[0][:back], -x[0][back:]))
    b.held = [back]
    b.new = [75 - back]
    b.append_new(binding, cache)
    _check_all(b, cache, [75])


def test_reading_the_last_tokens_only():
    b = kv_ref.Batch([0] * 3, [100, 33, 64], 2, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    k, v = _read(b, cache, [71, 33, 50], [29, 0, 14])
    for got, raw in ((k, b.k_all), (v, b.v_all)):
        want = torch.cat([kv_ref.held_values(raw[0], 16)[71:], kv_ref.held_values(raw[2], 16)[50:]])
        assert torch.equal(got.cpu(), want)


def test_padding_and_numbers_outside_are_left_alone():
    P, D, kv = 16, 64, 2
    b = kv_ref.Batch([20, 5, 40, 0, 9], [1] * 5, kv, D, P)
    cache = b.cache(binding)
    before = [t.clone() for t in (cache.codes, cache.scales, cache.tails, cache.tail_scales)]
    table, lens, slots, _ = b.args()
    k, v = b.cut(b.k_all, b.held, b.new), b.cut(b.v_all, b.held, b.new)
    for bad_slots, bad_lens in (([-1] * 5, b.held), (slots.tolist(), [-1] * 5), ([7] * 5, b.held),
                                (slots.tolist(), [table.shape[1] * P] * 5)):
        binding.kv_append(cache, k, v, table, b.ints(bad_lens), b.ints(bad_slots))
        out = torch.full((5, kv, D), 7.0, device="cuda")
        binding.kv_read(cache, table, b.ints(bad_lens), b.ints(bad_slots), out=(out, out.clone()))
        assert (out == 7.0).all()
    # a page outside the cache takes nothing
    full = b.args([15] * 5)[1]
    for page in (-1, b.pages, 2 ** 31 - 1):
        binding.kv_append(cache, k, v, torch.full_like(table, page), full, b.ints([6] * 5)[:5])
    for t, old in zip((cache.codes, cache.scales), before):
        assert torch.equal(t, old)
    # cu outside the call's tokens
    for cu in ([9, 9, 9, 9, 9, 9], [-3, -3, -2, -2, -2, -2], [5, 4, 3, 2, 1, 0]):
        binding.kv_append(cache, k, v, table, lens, slots, cu=b.ints(cu))
    for t, old in zip((cache.codes, cache.scales), before):
        assert torch.equal(t, old)


def test_rows_behind_the_last_sequence_stay():
    b = kv_ref.Batch([0, 0], [20, 3], 2, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    table, lens, slots, cu = b.args()
    k = torch.full((40, 2, 64), 3.0, device="cuda", dtype=torch.float16)
    v = k.clone()
    binding.kv_read(cache, table, lens, slots, cu=cu, tokens=40, out=(k, v))
    assert (k[23:] == 3.0).all() and (v[23:] == 3.0).all() and not (k[:23] == 3.0).all()


def test_tokens_behind_the_table_are_dropped():
    P = 16
    b = kv_ref.Batch([0], [3 * P + 5], 1, 64, P, spare=0)
    cache = b.cache(binding)
    table, lens, slots, cu = b.args()
    binding.kv_append(cache, b.k_all[0].cuda(), b.v_all[0].cuda(), table[:, :3], lens, slots, cu=cu)
    _check_all(b, cache, [3 * P])
    assert (cache.tails == 0).all()


# --- sequences that continue others -------------------------------------------------

@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 128), (192, 32)])
def test_fork_and_both_go_on(D, P):
    held = [P + 3, 2 * P, 7, 0, 3 * P + P // 2 + 1]
    b = kv_ref.Batch(held + [0] * 5, [P] * 10, 3, D, P, spare=5)
    cache = b.cache(binding)
    for i in range(5):  # what a fork holds is its parent's
        b.k_all[5 + i] = torch.cat((b.k_all[i][:held[i]], b.k_all[5 + i][:P]))
        b.v_all[5 + i] = torch.cat((b.v_all[i][:held[i]], b.v_all[5 + i][:P]))
    own = b.table_cpu.clone()
    table, lens, slots, _ = b.args(held + [0] * 5)
    # the fork's own pages behind the shared ones, from the parent's spare entries
    free = [p for p in range(b.pages) if p not in set(own.flatten().tolist())]
    codes = cache.codes.clone()
    binding.kv_fork(cache, table, lens, slots, b.ints([0, 1, 2, 3, 4]), b.ints([5, 6, 7, 8, 9]))
    assert lens.tolist() == held + held
    for i in range(5):
        full = held[i] // P
        assert table[5 + i, :full].tolist() == own[i, :full].tolist()
        assert table[5 + i, full:].tolist() == own[5 + i, full:].tolist()
    assert torch.equal(cache.codes, codes) and len(free) > 0
    # the fork's page for its first new page: the one it had at entry 0 moves behind the shared ones
    t = table.cpu()
    for i in range(5):
        t[5 + i, held[i] // P] = own[5 + i, 0]
        t[5 + i, held[i] // P + 1:] = -1
    b.table_cpu = t
    b.held, b.new = held + held, [P] * 10
    b.append_new(binding, cache)
    # (a second incomplete page has no page of its own yet: its tokens are in the tail)
    _check_all(b, cache, [h + P for h in held + held])


def test_fork_refuses_numbers_outside_on_the_device():
    b = kv_ref.Batch([20, 9, 0], [1] * 3, 2, 64, 16)
    cache = b.cache(binding)
    table, lens, slots, _ = b.args()
    tails, t0 = cache.tails.clone(), table.clone()
    binding.kv_fork(cache, table, lens, slots, b.ints([0, -1, 3, 1, 5]), b.ints([3, 2, 2, 1, -7]))
    assert torch.equal(cache.tails, tails) and torch.equal(table, t0) and lens.tolist() == [20, 9, 0]
    binding.kv_fork(cache, table, b.ints([20, -1, 10 ** 6]), slots, b.ints([1, 2]), b.ints([0, 0])[:2])
    assert torch.equal(cache.tails, tails) and torch.equal(table, t0)
    # slots outside: the row is copied, the tokens have nowhere to go
    binding.kv_fork(cache, table, lens, b.ints([-1, 0, 99]), b.ints([0]), b.ints([2]))
    assert torch.equal(cache.tails, tails) and lens.tolist() == [20, 9, 20]


def test_no_pairs_and_no_entries():
    b = kv_ref.Batch([20], [1], 2, 64, 16)
    cache = b.cache(binding)
    table, lens, slots, _ = b.args()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    binding.kv_fork(cache, table, lens, slots, none, none)
    binding.kv_fork(cache, table[:0], none, none, b.ints([0]), b.ints([1]))
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    binding.kv_append(cache, empty, empty, table[:0], none, none)
    binding.kv_append(cache, empty, empty, table, lens, slots, cu=b.ints([0, 0]))
    k, v = binding.kv_read(cache, table, lens, slots, cu=b.ints([0, 0]), tokens=0)
    assert k.shape == v.shape == (0, 2, 64)


def test_offsets_past_32_bits():
    """Codes and tails of more than 2^32 bytes: the pages and slots at their far ends."""
    P, D, kv = 64, 128, 8
    pages, slots_n = 34000, 17000  # 4.5 GB of codes, 4.5 GB of tails
    cache = binding.KvCache(pages, slots_n, kv, D, page_size=P)
    b = kv_ref.Batch([0, 0], [2 * P + 9, P + 1], kv, D, P, spare=0)
    b.pages = pages
    b.table_cpu = torch.tensor([[pages - 1, 3, 0], [pages - 2, 0, 0]], dtype=torch.int32)
    b.slots_cpu = torch.tensor([slots_n - 1, slots_n - 2], dtype=torch.int32)
    b.append_new(binding, cache)
    _check_all(b, cache, b.new)
    assert (cache.codes[pages - 1] != 0).any() and (cache.tails[slots_n - 1] != 0).any()
    q = torch.randn((2, 16, D), generator=b.gen).to(torch.bfloat16).cuda()
    held = [n - 1 for n in b.new]
    table, lens, slots, _ = b.args(held, [1, 1])
    out = binding.kv_attention(cache, q, table, lens, slots)
    for i in range(2):
        want, far = kv_ref.attention(q[i:i + 1], kv_ref.held_values(b.k_all[i], P), kv_ref.held_values(b.v_all[i], P),
                                     held[i], D ** -0.5)
        kv_ref.check(out[i:i + 1], want, far)
    chunk = torch.randn((P, 16, D), generator=b.gen).to(torch.bfloat16).cuda()
    table, lens, slots, cu = b.args([b.new[0] - P, 0], [P, 0])
    out = binding.kv_attention(cache, chunk, table, lens, slots, cu=cu)
    want, far = kv_ref.attention(chunk, kv_ref.held_values(b.k_all[0], P), kv_ref.held_values(b.v_all[0], P),
                                 b.new[0] - P, D ** -0.5)
    kv_ref.check(out, want, far)
    src, dst = b.ints([0]), b.ints([1])
    binding.kv_fork(cache, table, b.ints(b.new), slots, src, dst)
    assert torch.equal(cache.tails[slots_n - 1, :, :, :16 * D], cache.tails[slots_n - 2, :, :, :16 * D])
    del cache
    torch.cuda.empty_cache()
