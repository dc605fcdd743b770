"""The attention block and a decoder layer of both blocks: prompts, then tokens, against the same steps by the entry
points and the attention's formula in 64 bits."""
import pytest
import torch

from nvfp4_token_quant_amd import binding, synth
from nvfp4_token_quant_amd.block import AttentionBlock, DecoderLayer, MoeBlock
from tests import kv_ref
from tests.layer_fixtures import gpu_weights

pytestmark = pytest.mark.gpu

D, KV, G, P = 64, 2, 3, 16
HEADS = KV * G


def _randn(*shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).cuda()


def _block(H, window=0, after=True):
    wqkv, sqkv = binding.int8_quantize_per_token(_randn((HEADS + 2 * KV) * D, H, seed=1, scale=H ** -0.5))
    wo, so = binding.int8_quantize_per_token(_randn(H, HEADS * D, seed=2, scale=(HEADS * D) ** -0.5))
    cache = binding.KvCache(40, 6, KV, D, page_size=P)
    norm = lambda s: binding.Norm((1 + 0.1 * _randn(H, seed=s)).bfloat16())  # noqa: E731
    return AttentionBlock(cache, HEADS, wqkv, sqkv, wo, so, norm(3), norm(4) if after else None, window=window,
                          qkv_bias=_randn((HEADS + 2 * KV) * D, seed=5, scale=0.1), res_scale=0.9, out_scale=1.1)


def _layer(H):
    L = synth.LAYERS[1]
    layer = binding.MoeLayer(64, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(1))
    codes, scale = binding.int8_quantize_per_token(_randn(L.E, H, seed=6, scale=H ** -0.5))
    return MoeBlock(layer, codes, scale, binding.Norm((1 + 0.1 * _randn(H, seed=7)).bfloat16()))


def _steps():
    """A prompt of two sequences, single tokens, a mixed step, the same with a padding entry."""
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.randperm(40, generator=torch.Generator().manual_seed(0), dtype=torch.int32).cuda()[:36].view(3, 12).contiguous()
    slots = ints([4, 0, 2])
    return table, slots, [([0, 0, 0], [30, 0, 17]), ([30, 0, 17], None), ([31, 1, 18], [1, 20, 1])]


@pytest.mark.parametrize("window", [0, 9])
def test_block_is_its_operators(window):
    H = 256
    block, twin = _block(H, window), _block(H, window)
    table, slots, steps = _steps()
    seen_k, seen_v = [[] for _ in range(3)], [[] for _ in range(3)]
    nxt = binding.Norm()
    for held, new in steps:
        n = [1, 1, 1] if new is None else new
        cu = None if new is None else torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        lens = torch.tensor(held, dtype=torch.int32, device="cuda")
        r = _randn(sum(n), H, seed=sum(held)).bfloat16()
        r2, h2 = block.forward(r, table, lens, slots, cu, next_before=nxt)
        # by the entry points
        h = torch.empty_like(r)
        _, h = binding.block_norm(r, before=twin.before, h_out=h)
        qkv = binding.int8_linear(h, twin.qkv_codes, twin.qkv_scale, bias=twin.qkv_bias).view(sum(n), HEADS + 2 * KV, D)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        binding.kv_append(twin.cache, k, v, table, lens, slots, cu=cu)
        o = binding.kv_attention(twin.cache, q, table, lens, slots, cu=cu, window=window)
        y = binding.int8_linear(o.view(sum(n), HEADS * D), twin.out_codes, twin.out_scale_w)
        want = binding.block_norm(r, y, before=nxt, after=twin.after, res_scale=0.9, out_scale=1.1)
        assert torch.equal(r2, want[0]) and torch.equal(h2, want[1])
        if new is None or not any(held):  # the same step again leaves what it found
            given = block.forward(r, table, lens, slots, cu, h=h, next_before=nxt)
            assert torch.equal(given[0], r2) and torch.equal(given[1], h2)
        # the attention by its formula, over all tokens so far
        at = 0
        for i in range(3):
            seen_k[i].append(k[at:at + n[i]].cpu())
            seen_v[i].append(v[at:at + n[i]].cpu())
            kk, vv = (kv_ref.held_values(torch.cat(x[i]), P) for x in (seen_k, seen_v))
            if n[i]:
                kv_ref.check(o[at:at + n[i]], *kv_ref.attention(q[at:at + n[i]], kk, vv, held[i], D ** -0.5, window))
            at += n[i]


def test_decoder_layer():
    H = synth.LAYERS[1].H
    att, moe = _block(H, after=False), _layer(H)
    layer = DecoderLayer(att, moe)
    twin = _block(H, after=False)
    table, slots, steps = _steps()
    nxt = binding.Norm()
    for held, new in steps:
        n = [1, 1, 1] if new is None else new
        cu = None if new is None else torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        lens = torch.tensor(held, dtype=torch.int32, device="cuda")
        r = _randn(sum(n), H, seed=3 + sum(held))
        out, h = layer.forward(r, table, lens, slots, cu, next_before=nxt)
        r1, h1 = twin.forward(r, table, lens, slots, cu, next_before=moe.before)
        want = moe.forward(r1, h=h1, next_before=nxt)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(h, want[1]) and torch.isfinite(out).all()


def test_a_captured_layer_step():
    """A decode step of the whole layer in one graph, replayed while the sequences grow, one entry padding."""
    H = synth.LAYERS[1].H
    layer, twin = DecoderLayer(_block(H), _layer(H)), _block(H)
    ref = DecoderLayer(twin, layer.moe)
    table, slots, _ = _steps()
    slots[1] = -1
    lens = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    r = torch.zeros((3, H), device="cuda")
    layer.forward(r, table, lens, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = layer.forward(r, table, lens, slots)
    live = [0, 2]
    for i in range(20):
        r.copy_(_randn(3, H, seed=100 + i))
        g.replay()
        got = out[live].clone()
        want, _ = ref.forward(r, table, lens, slots)
        torch.cuda.synchronize()
        assert torch.equal(got, want[live])
        lens += 1


def test_refusals():
    cache = binding.KvCache(4, 2, KV, D, page_size=P)
    codes = lambda r, c: torch.zeros((r, c), dtype=torch.int8, device="cuda")  # noqa: E731
    s = torch.ones(1024, device="cuda")
    norm = binding.Norm()
    for heads, qkv, out in ((5, (9 * D, 128), (128, 5 * D)), (0, (4 * D, 128), (128, 0)), (6, (9 * D, 128), (128, 6 * D)),
                            (6, (10 * D, 128), (128, 5 * D)), (6, (10 * D, 64), (128, 6 * D))):
        with pytest.raises(ValueError):
            AttentionBlock(cache, heads, codes(*qkv), s, codes(*out), s, norm)
