"""The key-value cache's operators called as programs call them: in captured and replayed steps, on other streams,
from two threads, with tensors that they refuse."""
import threading

import pytest
import torch

from nvfp4_token_quant_amd import binding
from tests import kv_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,D,G,start", [(16, 64, 4, 13), (64, 128, 8, 2040)])
def test_a_captured_decode_step_goes_on(P, D, G, start):
    """One graph of append, attention and read is replayed token by token, over the ends of pages and past the
    length where a sequence is cut into pieces, beside the same steps run eagerly on a second cache."""
    steps = 12
    held = [start, start + 3, 0, 5]
    b = kv_ref.Batch(held, [steps] * 4, 2, D, P, spare=3)
    caches = [b.cache(binding), b.cache(binding)]
    table, lens, slots, _ = b.args()
    k, v = (torch.zeros((4, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((4, 2 * G, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    back = [torch.zeros((4, 2, D), device="cuda") for _ in range(2)]

    def step(cache, out, back):
        binding.kv_append(cache, k, v, table, lens, slots)
        binding.kv_attention(cache, q, table, lens, slots, out=out)
        binding.kv_read(cache, table, lens, slots, out=back)

    graph = torch.cuda.CUDAGraph()
    step(caches[0], out, back)  # (the first token's step, run again by the first replay)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(caches[0], out, back)
    eager, eager_back = torch.zeros_like(q), [torch.zeros_like(t) for t in back]
    queries = (torch.randn((steps, 4, 2 * G, D), generator=b.gen)).to(torch.bfloat16).cuda()
    ks = [torch.stack([x[h + i] for x, h in zip(b.k_all, held)]).cuda() for i in range(steps)]
    vs = [torch.stack([x[h + i] for x, h in zip(b.v_all, held)]).cuda() for i in range(steps)]
    for i in range(steps):
        k.copy_(ks[i])
        v.copy_(vs[i])
        q.copy_(queries[i])
        graph.replay()
        if i % 3 == 1:
            torch.cuda.synchronize()
        step(caches[1], eager, eager_back)
        assert torch.equal(out, eager)
        assert all(torch.equal(x, y) for x, y in zip(back, eager_back))
        lens += 1
    full = [h + steps for h in held]
    want, far = kv_ref.attention(queries[-1, :1], kv_ref.held_values(b.k_all[0], P), kv_ref.held_values(b.v_all[0], P),
                                 full[0] - 1, D ** -0.5)
    kv_ref.check(out[:1], want, far)


def test_two_graphs_that_share_a_cache():
    """Graphs of two batches, each with its own workspace, replayed in turn and together."""
    b = kv_ref.Batch([3000, 2500], [1, 1], 2, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(8)
    table, lens, slots, _ = b.args()
    want = binding.kv_attention(cache, q, table, lens, slots)
    graphs, outs, keep = [], [], []
    for i in range(2):
        part = [q[i:i + 1].contiguous(), table[i:i + 1], lens[i:i + 1], slots[i:i + 1]]
        keep.append(part)
        outs.append(torch.zeros_like(part[0]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.kv_attention(cache, part[0], *part[1:], out=outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ref, far = b.attention(q)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        kv_ref.check(torch.cat(outs), ref, far)
    kv_ref.check(want, ref, far)


def test_on_another_stream():
    b = kv_ref.Batch([100, 30], [40, 1], 2, 128, 32)
    cache = b.cache(binding)
    k, v = b.cut(b.k_all, b.held, b.new), b.cut(b.v_all, b.held, b.new)
    q = b.queries(4)
    args = b.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    binding.kv_append(cache, k, v, *args, stream=s)
    out = binding.kv_attention(cache, q, *args, stream=s)
    kk, vv = binding.kv_read(cache, *args, tokens=41, dtype=torch.float32, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want, far = b.attention(q)
    kv_ref.check(out, want, far)
    assert torch.equal(kk[-1].cpu(), kv_ref.held_values(b.k_all[1], 32)[-1])
    assert torch.equal(vv[-1].cpu(), kv_ref.held_values(b.v_all[1], 32)[-1])
    with pytest.raises(ValueError):
        binding.kv_attention(cache, q.cpu(), *args, stream=s)


def test_from_two_threads():
    b = kv_ref.Batch([3000, 200], [1, 1], 2, 64, 16)
    cache = b.cache(binding)
    b.append_new(binding, cache)
    q = b.queries(8)
    table, lens, slots, _ = b.args()
    want = binding.kv_attention(cache, q, table, lens, slots)
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not torch.equal(binding.kv_attention(cache, q, table, lens, slots), want):
                    bad.append(1)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def _refusals():
    b = kv_ref.Batch([20, 7], [1, 1], 2, 64, 16)
    cache = b.cache(binding)
    table, lens, slots, cu = b.args()
    k, v = b.cut(b.k_all, b.held, b.new), b.cut(b.v_all, b.held, b.new)
    q = b.queries(4)
    append = lambda k=k, v=v, table=table, lens=lens, slots=slots, cu=None, c=cache: (  # noqa: E731
        binding.kv_append(c, k, v, table, lens, slots, cu=cu))
    attention = lambda q=q, table=table, lens=lens, slots=slots, **kw: (  # noqa: E731
        binding.kv_attention(cache, q, table, lens, slots, **kw))
    read = lambda **kw: binding.kv_read(cache, table, lens, slots, **kw)  # noqa: E731
    fork = lambda s, d, **kw: binding.kv_fork(cache, kw.get("table", table), kw.get("lens", lens), slots, s, d)  # noqa: E731
    g = lambda t: t.float().requires_grad_().to(t.dtype)  # noqa: E731
    i64 = lambda t: t.long()  # noqa: E731
    two = b.ints([0, 1])
    return {
        "k gradient": lambda: append(k=g(k)), "v gradient": lambda: append(v=g(v)), "q gradient": lambda: attention(q=g(q)),
        "out gradient": lambda: attention(out=g(torch.empty_like(q))),
        "k f32": lambda: append(k=k.float(), v=v.float()), "q f32": lambda: attention(q=q.float()),
        "types differ": lambda: append(v=v.half()), "k on the host": lambda: append(k=k.cpu()),
        "k matrix": lambda: append(k=k.view(2, 128)), "k heads": lambda: append(k=k[:, :1]),
        "v tokens": lambda: append(v=v[:1]), "channel stride": lambda: append(k=k.transpose(1, 2).contiguous().transpose(1, 2)),
        "table type": lambda: append(table=i64(table)), "table vector": lambda: append(table=table[0]),
        "table strides": lambda: append(table=table.t().contiguous().t()), "lens type": lambda: append(lens=i64(lens)),
        "lens size": lambda: append(lens=lens[:1]), "lens none": lambda: append(lens=None),
        "slots on the host": lambda: append(slots=slots.cpu()), "cu size": lambda: append(cu=cu[:2]),
        "cu strides": lambda: append(cu=b.ints([0, 0, 1, 1, 2, 2])[::2]),
        "head_dim": lambda: attention(q=q[..., :32]), "out type": lambda: attention(out=torch.empty_like(q).half()),
        "out shape": lambda: attention(out=torch.empty_like(q)[:1]), "out list": lambda: read(out=[k]),
        "read type": lambda: read(dtype=torch.int8), "read tokens": lambda: read(cu=cu),
        "read out strides": lambda: read(out=(k.transpose(0, 1).contiguous().transpose(0, 1), v)),
        "read out types": lambda: read(out=(k, v.half())), "src type": lambda: fork(i64(two), two),
        "dst size": lambda: fork(two, two[:1]), "dst none": lambda: fork(two, None), "fork table": lambda: fork(two, two, table=i64(table)),
        "no cache": lambda: append(c=binding.Norm()),
    }


NAMES = ("k gradient", "v gradient", "q gradient", "out gradient", "k f32", "q f32", "types differ", "k on the host", "k matrix",
         "k heads", "v tokens", "channel stride", "table type", "table vector", "table strides", "lens type", "lens size",
         "lens none", "slots on the host", "cu size", "cu strides", "head_dim", "out type", "out shape", "out list",
         "read type", "read tokens", "read out strides", "read out types", "src type", "dst size", "dst none", "fork table",
         "no cache")


@pytest.mark.parametrize("name", NAMES)
def test_refused(name):
    call = _refusals()[name]
    with pytest.raises((ValueError, TypeError)):
        call()
    if name.endswith("gradient"):
        with torch.no_grad():
            call()
    torch.cuda.synchronize()


def test_all_refusals_are_tried():
    assert set(_refusals()) == set(NAMES)


def test_the_librarys_refusals_are_errors():
    b = kv_ref.Batch([20, 7], [1, 1], 2, 64, 16)
    cache = b.cache(binding)
    table, lens, slots, _ = b.args()
    q = b.queries(4)
    for call in (lambda: binding.kv_attention(cache, q[:, :3], table, lens, slots),
                 lambda: binding.kv_attention(cache, q, table, lens, slots, window=-1),
                 lambda: binding.kv_attention(cache, q, table, lens, slots, scale=float("nan")),
                 lambda: binding.kv_attention(cache, q, table, lens, slots, out=q),
                 lambda: binding.kv_attention(cache, q[:1], table, lens, slots),
                 lambda: binding.kv_attention(cache, torch.cat((q, q), 2)[..., 4:68], table, lens, slots)):
        with pytest.raises(binding.Nvfp4Error):
            call()
    torch.cuda.synchronize()
