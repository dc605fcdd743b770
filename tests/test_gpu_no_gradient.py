"""The operators around the layer have no gradient: a call whose result would need one is refused."""
import pytest
import torch

from nvfp4_token_quant_amd import binding

pytestmark = pytest.mark.gpu


def _calls():
    x = torch.randn((4, 64), device="cuda")
    w, ws = binding.int8_quantize_per_token(torch.randn((32, 64), device="cuda"))
    b, v = torch.randn(32, device="cuda"), torch.randn(64, device="cuda")
    q, s = binding.int8_quantize_per_token(x)
    g = lambda t: t.clone().requires_grad_()  # noqa: E731
    return {
        "logits": lambda: binding.route(g(x), 4, binding.Router()),
        "balance bias": lambda: binding.route(x, 4, binding.Router(), bias=g(v)),
        "residual": lambda: binding.block_norm(g(x), x, before=binding.Norm(v)),
        "y": lambda: binding.block_norm(x, g(x), before=binding.Norm(v)),
        "weight": lambda: binding.block_norm(x, x, before=binding.Norm(torch.nn.Parameter(v))),
        "norm bias": lambda: binding.block_norm(x, x, after=binding.Norm(v, g(v))),
        "gate": lambda: binding.block_norm(x, x, gate=g(v)),
        "token gate": lambda: binding.block_norm(x, x, gate=g(x[:, :1])),
        "quantized": lambda: binding.int8_quantize_per_token(g(x)),
        "scale": lambda: binding.int8_matmul(q, g(s), w, ws),
        "channel scale": lambda: binding.int8_matmul(q, s, w, g(ws)),
        "bias": lambda: binding.int8_matmul(q, s, w, ws, bias=g(b)),
        "x": lambda: binding.int8_linear(g(x), w, ws),
        "linear bias": lambda: binding.int8_linear(x, w, ws, bias=g(b)),
        "out": lambda: binding.int8_linear(x, w, ws, out=g(torch.empty((4, 32), device="cuda"))),
    }


NAMES = ("logits", "balance bias", "residual", "y", "weight", "norm bias", "gate", "token gate", "quantized", "scale",
         "channel scale", "bias", "x", "linear bias", "out")


@pytest.mark.parametrize("name", NAMES)
def test_no_gradient_is_cut_without_a_word(name):
    call = _calls()[name]
    with pytest.raises(ValueError, match="gradient"):
        call()
    with torch.no_grad():
        call()
    with torch.inference_mode():
        call()
    torch.cuda.synchronize()


def test_all_names_are_tried():
    assert set(_calls()) == set(NAMES)
