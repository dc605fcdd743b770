"""The layer with its router set, and the operators of a block run together."""
import threading

import numpy as np
import pytest
import torch

import oracle
from nvfp4_token_quant_amd import binding, synth
from nvfp4_token_quant_amd.block import MoeBlock
from tests import ops_ref
from tests.layer_fixtures import (bf16_tensor_to_f64, check_layer_tolerance, gpu_weights, oracle_weights,
                                  to_device_bf16)

pytestmark = pytest.mark.gpu


def _bias(E):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()


# every prologue of the forward: one block (T <= 64), small batches, routing blocks, the three-kernel schedule
@pytest.mark.parametrize("layer_id,T,groups,top_groups,best", [
    (1, 3, 4, 2, 2), (1, 16, 1, 1, 1), (1, 100, 4, 2, 1), (1, 300, 2, 1, 2), (2, 64, 8, 4, 2), (7, 33, 6, 3, 2),
    (7, 300, 10, 5, 1), (10, 8, 8, 4, 2), (11, 129, 8, 4, 2)])
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("softmax", False)])
def test_layer_with_router(layer_id, T, groups, top_groups, best, score, bias):
    L = synth.LAYERS[layer_id]
    print(f"layer {layer_id} T={T} router {score} bias={bias} groups={groups}", flush=True)
    rule = dict(score=score, groups=groups, top_groups=top_groups, group_best=best, renormalize=bias, scale=1.5)
    b = _bias(L.E) if bias else None
    x = synth.activations(layer_id, T)
    logits = torch.from_numpy(synth.router_logits(layer_id, T)).cuda()
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(layer_id))
    xt = to_device_bf16(x)
    before = layer.forward(xt, logits)
    layer.set_router(binding.Router(**rule), b)
    out = layer.forward(xt, logits)
    torch.cuda.synchronize()
    ids = layer.read_buffer("TOPK_IDS", torch.int32, (T, L.k))
    w = layer.read_buffer("TOPK_W", torch.float32, (T, L.k))
    alone = binding.route(logits, L.k, binding.Router(**rule), bias=b)
    assert torch.equal(ids, alone[0]) and torch.equal(w, alone[1])
    oids, _ = ops_ref.route(logits, L.k, bias=b, **rule)
    np.testing.assert_array_equal(ids.cpu().numpy(), oids)
    oids, ow = ids.cpu().numpy(), w.cpu().numpy()
    counts, offsets, perm, inv = oracle.permute(oids, L.E)
    np.testing.assert_array_equal(layer.read_buffer("PERM", torch.int32, (T * L.k,)).cpu().numpy(), perm)
    np.testing.assert_array_equal(layer.read_buffer("INV", torch.int32, (T * L.k,)).cpu().numpy(), inv)
    ref = oracle.moe_layer(x, oids, ow, np.arange(T), L.H, L.I, oracle_weights(layer_id, np.unique(oids)))
    check_layer_tolerance(bf16_tensor_to_f64(out), ref)
    layer.set_router(None)
    again = layer.forward(xt, logits)
    torch.cuda.synchronize()
    assert torch.equal(again, before)
    layer.close()


def test_router_bias_in_place_in_a_graph():
    L = synth.LAYERS[1]
    T = 40
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(1))
    x = to_device_bf16(synth.activations(1, T))
    logits = torch.from_numpy(synth.router_logits(1, T)).cuda()
    r = binding.Router(score="sigmoid", groups=4, top_groups=2, group_best=2)
    layer.set_router(r, torch.zeros(L.E, device="cuda"))
    out = torch.empty_like(x)
    layer.forward_into(x, logits, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            layer.forward_into(x, logits, out)
    torch.cuda.synchronize()
    seen = []
    for i in range(3):
        layer.set_router(r, i * _bias(L.E))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        layer.forward_into(x, logits, out)
        torch.cuda.synchronize()
        assert torch.equal(out, got)
        seen.append(got)
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    with pytest.raises(binding.Nvfp4Error):
        layer.set_router(binding.Router(groups=3))
    with pytest.raises(binding.Nvfp4Error):
        layer.set_router(None, _bias(L.E))
    with pytest.raises(ValueError):
        layer.set_router(r, _bias(L.E + 1))
    layer.close()


@pytest.mark.parametrize("T", [30, 300])
def test_router_with_the_other_forwards(T):
    """Handed-over codes give the forward's output bit for bit with a router too; W4A16 takes the same routing."""
    L = synth.LAYERS[1]
    x = to_device_bf16(synth.activations(1, T))
    logits = torch.from_numpy(synth.router_logits(1, T)).cuda()
    rule, b = dict(score="sigmoid", groups=4, top_groups=3, group_best=2, scale=2.0), _bias(L.E)
    ids, w = binding.route(logits, L.k, binding.Router(**rule), bias=b)
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(1))
    layer.set_router(binding.Router(**rule), b)
    out = layer.forward(x, logits)
    again = layer.forward_quantized(*binding.quantize_per_token(x), logits)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    layer.close()
    wide = binding.MoeLayer(T, L.H, L.I, L.E, L.k, False, w4a16=True)
    wide.bind(gpu_weights(1))
    wide.set_router(binding.Router(**rule), b)
    wide.forward(x, logits)
    torch.cuda.synchronize()
    assert torch.equal(wide.read_buffer("TOPK_IDS", torch.int32, (T, L.k)), ids)
    assert torch.equal(wide.read_buffer("TOPK_W", torch.float32, (T, L.k)), w)
    wide.close()


def test_masked_tokens_and_shared_expert():
    """A token without any open expert gets only the shared expert's output."""
    L = synth.LAYERS[1]
    T = 12
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True, shared_expert="sum")
    layer.bind(gpu_weights(1, n_experts=L.E + 1))
    x = to_device_bf16(synth.activations(1, T))
    logits = torch.from_numpy(synth.router_logits(1, T)).cuda()
    logits[5] = -float("inf")
    layer.set_router(binding.Router(score="sigmoid", groups=4, top_groups=2))
    out = layer.forward(x, logits)
    layer.set_router(binding.Router(score="sigmoid", scale=0.0))
    shared = layer.forward(x, logits)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
    assert torch.equal(out[5], shared[5]) and not torch.equal(out[4], shared[4])
    layer.close()


@pytest.mark.parametrize("layer_id,T,residual", [(1, 1, torch.bfloat16), (1, 16, torch.float32), (2, 64, torch.float32),
                                                 (1, 300, torch.bfloat16)])
def test_block(layer_id, T, residual):
    """norm, 8-bit router projection, routing, experts, norm with gate and
    residual: each step against its reference on the step's own input."""
    L = synth.LAYERS[layer_id]
    print(f"block layer {layer_id} T={T} {residual}", flush=True)
    g = torch.Generator().manual_seed(T)

    def vec(scale=0.2, shift=1.0):
        return (scale * torch.randn(L.H, generator=g) + shift).to(torch.bfloat16).cuda()

    ws = [vec(), vec(), vec()]
    before, after, nxt = (binding.Norm(w, eps=1e-5) for w in ws)
    gate = vec(0.1, 0.5)
    wg, sg = binding.int8_quantize_per_token((torch.randn((L.E, L.H), generator=g) * L.H ** -0.5 * 2).cuda())
    layer = binding.MoeLayer(T, L.H, L.I, L.E, L.k, True)
    layer.bind(gpu_weights(layer_id))
    rule, b = dict(score="sigmoid", groups=4, top_groups=2, group_best=2, scale=1.5), _bias(L.E)
    layer.set_router(binding.Router(**rule), b)
    block = MoeBlock(layer, wg, sg, before, after=after, gate=gate, res_scale=1.0, out_scale=0.5)
    r = (2.0 * torch.randn((T, L.H), generator=g)).to(residual).cuda()
    r0 = r.clone()
    out, h2 = block.forward(r, next_before=nxt)
    torch.cuda.synchronize()
    assert torch.equal(r, r0) and out.dtype == residual and h2.dtype == torch.bfloat16
    h = torch.empty((T, L.H), dtype=torch.bfloat16, device="cuda")
    binding.block_norm(r, before=before, h_out=h)
    refs = [(ops_ref.f64(w), None, "rms", 1e-5, 0.0) for w in ws]
    _, _, rh, hs = ops_ref.block_norm(r, None, before=refs[0])
    ops_ref.check_norm(h, rh, hs)
    logits = block.logits(h)
    ops_ref.check_product(logits, *ops_ref.int8_product(*ops_ref.int8_rows(h), wg.cpu().numpy(), sg.cpu().numpy()))
    ids, w = ops_ref.route(logits, L.k, bias=b, **rule)
    y = layer.forward(h, logits)
    ref = oracle.moe_layer(h.view(torch.int16).cpu().numpy().view(np.uint16), ids.astype(np.int32), w.astype(np.float32),
                           np.arange(T), L.H, L.I, oracle_weights(layer_id, np.unique(ids)))
    check_layer_tolerance(bf16_tensor_to_f64(y), ref)
    want, size, wh, whs = ops_ref.block_norm(r, y, before=refs[2], after=refs[1], gate=gate, out_scale=0.5)
    ops_ref.check_norm(out, want, size)
    ops_ref.check_norm(h2, wh, whs)
    none = block.forward(r[:0], next_before=nxt)
    assert none[0].shape == (0, L.H) and none[1].shape == (0, L.H)
    # the next block takes the h that this pass gave
    again = block.forward(out, h=h2)
    torch.cuda.synchronize()
    assert again[1] is None and torch.isfinite(again[0].float()).all()
    # the whole block captured and replayed
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            cap = block.forward(r, next_before=nxt)
    for i in range(3):
        r.copy_((2.0 + i) * r0)
        graph.replay()
        torch.cuda.synchronize()
        eager = block.forward(r, next_before=nxt)
        torch.cuda.synchronize()
        assert torch.equal(cap[0], eager[0]) and torch.equal(cap[1], eager[1])
    layer.close()


def test_calls_from_two_threads():
    """The operators called from two threads at once, each on its own stream, one norm shared by both."""
    g = torch.Generator().manual_seed(11)
    x = [torch.randn((5, 640), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    l = [torch.randn((9, 96), generator=g).cuda() for _ in range(2)]
    w, ws = binding.int8_quantize_per_token(torch.randn((200, 640), generator=g).cuda())
    n = binding.Norm(torch.randn(640, generator=g).to(torch.bfloat16).cuda())
    rule = binding.Router(groups=4, top_groups=2)

    def calls(i):
        return (*binding.block_norm(x[i], x[1 - i], before=n, after=n), *binding.route(l[i], 6, rule),
                binding.int8_linear(x[i], w, ws), *binding.int8_quantize_per_token(x[i]))

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got = calls(i)
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(f"results of thread {i}")
        except Exception as e:  # reported below, in the main thread
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_results_allocated_under_capture():
    """A graph whose calls make their own results, replayed with eager calls between."""
    x = torch.randn((4, 512), generator=torch.Generator().manual_seed(12)).to(torch.bfloat16).cuda()
    w, ws = binding.int8_quantize_per_token(torch.randn((64, 512), generator=torch.Generator().manual_seed(13)).cuda())
    n, rule = binding.Norm(kind="layer"), binding.Router(score="sigmoid")

    def chain():
        r, h = binding.block_norm(x, x, before=n)
        logits = binding.int8_linear(h, w, ws, out_dtype=torch.float32)
        q, s = binding.int8_quantize_per_token(h)
        return r, h, logits, *binding.route(logits, 4, rule), binding.int8_matmul(q, s, w, ws, out_dtype=torch.float32)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = chain()
    for i in range(3):
        x.copy_(torch.randn((4, 512), generator=torch.Generator().manual_seed(20 + i)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(made, chain()):
            assert torch.equal(a, b)
        assert torch.equal(made[2], made[5])
