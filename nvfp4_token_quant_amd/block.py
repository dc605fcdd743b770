"""The mixture-of-experts block of a decoder around binding.MoeLayer.

    h      = before(r)                                  norm in front
    logits = 8-bit linear product of h                  router projection
    y      = experts(h, logits)                         routing and experts
    r'     = res_scale r + out_scale act(gate) after(y) norm behind, gate, residual
    h'     = next(r')                                   the next block's norm, in the same pass

[P3] (sglang PR #36624 summary), Cohere2MoeDecoderLayer.forward and
Cohere2MoeSparseMoeBlock.forward: input_layernorm, gate, topk and experts
around a residual stream.
"""
from __future__ import annotations

import torch

from . import binding


class MoeBlock:
    """layer: a MoeLayer with weights bound (and its router set, if not the
    default rule).  gate_codes int8 [E, H] and gate_scale f32 [E]: the
    router projection's weights, quantized per expert
    (binding.int8_quantize_per_token).  before / after: binding.Norm (after
    may be None).  gate, gate_sigmoid, res_scale, out_scale: as in
    binding.block_norm."""

    def __init__(self, layer, gate_codes, gate_scale, before, after=None, gate=None, gate_sigmoid=False,
                 res_scale=1.0, out_scale=1.0):
        if tuple(gate_codes.shape) != (layer.cfg.num_experts, layer.cfg.hidden):
            raise ValueError(f"gate_codes must be [{layer.cfg.num_experts}, {layer.cfg.hidden}], "
                             f"got {tuple(gate_codes.shape)}")
        self.layer, self.gate_codes, self.gate_scale = layer, gate_codes, gate_scale
        self.before, self.after, self.gate, self.gate_sigmoid = before, after, gate, gate_sigmoid
        self.res_scale, self.out_scale = res_scale, out_scale

    def logits(self, h):
        """Router logits f32 [T, E] of the normed hidden states."""
        return binding.int8_linear(h, self.gate_codes, self.gate_scale, out_dtype=torch.float32)

    def forward(self, residual, h=None, next_before=None):
        """residual [T, H], bf16 or f32; h bf16 [T, H]: before(residual) if the
        pass that made the residual gave it already (that pass normed the
        residual before rounding it, so with a bf16 residual the two differ by
        that rounding).  -> (r', h'), h' None without `next_before` (a
        binding.Norm)."""
        if h is None:
            h = torch.empty(residual.shape, dtype=torch.bfloat16, device=residual.device)
            _, h = binding.block_norm(residual, before=self.before, h_out=h)
        y = self.layer.forward(h, self.logits(h))
        return binding.block_norm(residual, y, before=next_before, after=self.after, gate=self.gate,
                                  gate_sigmoid=self.gate_sigmoid, res_scale=self.res_scale,
                                  out_scale=self.out_scale)
