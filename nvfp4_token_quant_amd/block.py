"""The blocks of a decoder: attention over an 8-bit key-value cache, and the
mixture of experts around binding.MoeLayer.

Attention (AttentionBlock):

    h       = before(r)                                 norm in front
    q, k, v = 8-bit linear product of h                 one projection
    cache  <- k, v                                      into pages, full ones in 8 bits
    y       = 8-bit linear product of attention(q)      over the cache; output projection
    r'      = res_scale r + out_scale act(gate) after(y)
    h'      = next(r')                                  the experts' norm, in the same pass

Experts (MoeBlock):

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


class AttentionBlock:
    """cache: a KvCache, this block's.  qkv_codes int8 [(heads + 2 kv_heads) D, H],
    qkv_scale f32: the rows of the query heads, the key heads and the value heads,
    quantized per row (binding.int8_quantize_per_token); out_codes int8 [H, heads D],
    out_scale_w f32 [H].  qkv_bias / out_bias: f32 or None.  scale, window: as in
    binding.kv_attention; before / after / gate / gate_sigmoid / res_scale / out_scale:
    as in MoeBlock."""

    def __init__(self, cache, heads, qkv_codes, qkv_scale, out_codes, out_scale_w, before, after=None, qkv_bias=None,
                 out_bias=None, scale=None, window=0, gate=None, gate_sigmoid=False, res_scale=1.0, out_scale=1.0):
        D, kv = cache.head_dim, cache.kv_heads
        if heads < 1 or heads % kv:
            raise ValueError(f"heads must be a multiple of the cache's {kv}, got {heads}")
        H = out_codes.shape[0]
        if tuple(qkv_codes.shape) != ((heads + 2 * kv) * D, H) or out_codes.shape[1] != heads * D:
            raise ValueError(f"qkv_codes must be [{(heads + 2 * kv) * D}, H] and out_codes [H, {heads * D}], got "
                             f"{tuple(qkv_codes.shape)} and {tuple(out_codes.shape)}")
        self.cache, self.heads = cache, heads
        self.qkv_codes, self.qkv_scale, self.qkv_bias = qkv_codes, qkv_scale, qkv_bias
        self.out_codes, self.out_scale_w, self.out_bias = out_codes, out_scale_w, out_bias
        self.before, self.after, self.scale, self.window = before, after, scale, window
        self.gate, self.gate_sigmoid, self.res_scale, self.out_scale = gate, gate_sigmoid, res_scale, out_scale

    def attend(self, h, table, lens, slots, cu=None):
        """The step's keys and values into the cache and its attention, [T, H], for the
        normed hidden states h bf16 [T, H]."""
        kv, D = self.cache.kv_heads, self.cache.head_dim
        qkv = binding.int8_linear(h, self.qkv_codes, self.qkv_scale, bias=self.qkv_bias)
        qkv = qkv.view(h.shape[0], self.heads + 2 * kv, D)
        q, k, v = qkv[:, :self.heads], qkv[:, self.heads:self.heads + kv], qkv[:, self.heads + kv:]
        binding.kv_append(self.cache, k, v, table, lens, slots, cu=cu)
        o = binding.kv_attention(self.cache, q, table, lens, slots, cu=cu, scale=self.scale, window=self.window)
        return binding.int8_linear(o.view(h.shape[0], self.heads * D), self.out_codes, self.out_scale_w,
                                   bias=self.out_bias)

    def forward(self, residual, table, lens, slots, cu=None, h=None, next_before=None):
        """residual [T, H], bf16 or f32, of the step that table, lens, slots and cu
        describe (binding.KvCache's calls); h and next_before as in MoeBlock.forward.
        Rows of tokens that belong to no sequence mean nothing.  -> (r', h')."""
        if h is None:
            h = torch.empty(residual.shape, dtype=torch.bfloat16, device=residual.device)
            _, h = binding.block_norm(residual, before=self.before, h_out=h)
        y = self.attend(h, table, lens, slots, cu)
        return binding.block_norm(residual, y, before=next_before, after=self.after, gate=self.gate,
                                  gate_sigmoid=self.gate_sigmoid, res_scale=self.res_scale,
                                  out_scale=self.out_scale)


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


class DecoderLayer:
    """An AttentionBlock and the MoeBlock behind it: the pass that makes the residual
    between them norms it for the experts."""

    def __init__(self, attention, moe):
        self.attention, self.moe = attention, moe

    def forward(self, residual, table, lens, slots, cu=None, h=None, next_before=None):
        """As AttentionBlock.forward; next_before is the next layer's attention norm."""
        residual, h = self.attention.forward(residual, table, lens, slots, cu, h=h, next_before=self.moe.before)
        return self.moe.forward(residual, h=h, next_before=next_before)
