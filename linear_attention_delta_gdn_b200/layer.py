"""A Gated DeltaNet-2 layer around the operator: input projection, gate activations, the Gated Delta Rule-2,
output projection.

The pages name the layer's parts only as the operator plus "two additional per-channel gate computations"
(GitHub README method bullets; aiexpert.news article) next to KDA's channel-wise decay. This module takes the
plainest reading (the same as the library's gate kernels, ``gdn2_layer_gates_fwd``):

    z = x W_in  ->  q, k (L2-normalised per head), v, b = sigmoid, w = sigmoid, log_alpha = -softplus(z_a + a_bias)
    o, S_T = Gated Delta Rule-2 (q, k, v, log_alpha, b, w, S0)
    y = o W_out

The projections are plain GEMMs (cuBLAS through torch.matmul); the gate activations, the operator and their
backward run in the library's kernels. Short convolutions, output normalisation and gating, and the hybrid
sliding-window layers of the pages' models are not part of this reading.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding


class LayerGates(torch.autograd.Function):
    """Gate activations through the library's kernels (forward and backward)."""

    @staticmethod
    def forward(ctx, z, a_bias, Dk, Dv):
        z = z.contiguous()
        out = binding.gdn2_layer_gates_fwd(z, Dk, Dv, a_bias)
        ctx.save_for_backward(z, a_bias if a_bias is not None else torch.empty(0))
        ctx.has_bias, ctx.Dk, ctx.Dv = a_bias is not None, Dk, Dv
        return out

    @staticmethod
    def backward(ctx, dq, dk, dv, db, dw, dla):
        z, a_bias = ctx.saved_tensors
        a_bias = a_bias if ctx.has_bias else None
        grads = [g.contiguous() if g is not None else torch.zeros(z.shape[:3] + (D,), dtype=z.dtype, device=z.device)
                 for g, D in zip((dq, dk, dv, db, dw, dla), (ctx.Dk, ctx.Dk, ctx.Dv, ctx.Dk, ctx.Dv, ctx.Dk))]
        dz = binding.gdn2_layer_gates_bwd(z, *grads, ctx.Dk, ctx.Dv, a_bias)
        da = None
        if ctx.has_bias:   # the bias gradient: dz_a summed over batch and tokens
            da = dz[..., 3 * ctx.Dk + 2 * ctx.Dv:].float().sum((0, 1))
        return dz, da, None, None


class _Float32Parts(torch.nn.Module):
    """A module whose members named in ``_float32`` keep their 32 bits when it is cast (``.to(torch.bfloat16)`` and the like):
    the kernels take them in no other type, and a frequency or decay that has been through 8 bits is another one."""
    _float32 = ()

    def _apply(self, *args, **kwargs):
        before = {n: (t.detach(), None if t.grad is None else t.grad.detach())
                  for n in self._float32 for t in (getattr(self, n),) if t.dtype == torch.float32}
        super()._apply(*args, **kwargs)
        for n, (data, grad) in before.items():
            t = getattr(self, n)
            if t.dtype != torch.float32:   # cast: the same bits again, where the module now is
                t.grad = None
                t.data = data.to(t.device)
                t.grad = None if grad is None else grad.to(t.device)
        return self


class Gdn2Layer(_Float32Parts):
    """``y, S_T = layer(x, S0)`` for x [B, T, d_model]; bf16 (tensor-core operator path at d = 128) or fp32 (the projections'
    type, also by ``.to``; the decay bias stays float32)."""
    _float32 = ("a_bias",)

    def __init__(self, d_model: int, n_heads: int, d_k: int = 128, d_v: int = 128, chunk: int = 64,
                 dtype=torch.bfloat16, device=None, decay_bias: float = -4.0):
        super().__init__()
        self.d_model, self.H, self.Dk, self.Dv, self.chunk = d_model, n_heads, d_k, d_v, chunk
        width = n_heads * (4 * d_k + 2 * d_v)
        self.W_in = torch.nn.Parameter(torch.randn(d_model, width, device=device).div_(math.sqrt(d_model)).to(dtype))
        self.W_out = torch.nn.Parameter(torch.randn(n_heads * d_v, d_model, device=device)
                                        .div_(math.sqrt(n_heads * d_v)).to(dtype))
        # softplus(-4) ~ 0.018: a slow resting decay per token
        self.a_bias = torch.nn.Parameter(torch.full((n_heads, d_k), float(decay_bias), device=device))

    def forward(self, x, S0: Optional[torch.Tensor] = None):
        B, T, _ = x.shape
        z = (x @ self.W_in).view(B, T, self.H, 4 * self.Dk + 2 * self.Dv)
        q, k, v, b, w, la = LayerGates.apply(z, self.a_bias, self.Dk, self.Dv)
        o, ST = binding.gated_delta_rule2(q, k, v, la, b, w, S0, self.chunk)
        y = o.reshape(B, T, self.H * self.Dv) @ self.W_out
        return y, ST


class DecayLinearAttentionLayer(_Float32Parts):
    """A linear-attention layer with one fixed decay per head:

        q, k = x W_qk per head,  RMS-normalised with a weight each, pairs of channels turned by the token's position
        v = x W_v;   o, S_T = linear attention (q, k, v, log_decay, S0);   y = o W_out

    ``y, S_T = layer(x, S0, positions)`` for x [B, T, d_model], or packed [Ttot, d_model] with ``cu_seqlens`` and ``Tmax``;
    ``layer.step(x, positions, S, slots)`` for one token of each of B requests. ``pairs`` (d_k / 2 if not given) channel
    pairs turn; with ``sections`` pair by pair along several axes, positions then being [axes, ...]. ``log_decay`` [n_heads]
    defaults to memories of 8 to 256 tokens. bf16 or fp32: the projections' type, also by ``.to``; the norms' weights, decays
    and frequencies stay float32.
    """
    _float32 = ("q_weight", "k_weight", "log_decay", "inv_freq")

    def __init__(self, d_model: int, n_heads: int, d_k: int = 128, d_v: int = 128, pairs: Optional[int] = None, sections=None,
                 base: float = 10000.0, eps: float = 1e-6, log_decay: Optional[torch.Tensor] = None, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        self.d_model, self.H, self.Dk, self.Dv, self.eps = d_model, n_heads, d_k, d_v, eps
        pairs = pairs or (sum(sections) if sections else d_k // 2)
        if sections and sum(sections) != pairs:
            raise ValueError("sections %s do not add up to %d pairs" % (list(sections), pairs))
        rand = lambda m, n: torch.nn.Parameter(torch.randn(m, n, device=device).div_(math.sqrt(m)).to(dtype))
        self.W_qk, self.W_v, self.W_out = rand(d_model, 2 * n_heads * d_k), rand(d_model, n_heads * d_v), rand(n_heads * d_v, d_model)
        # products of normalised queries and keys start at a variance of one
        self.q_weight = torch.nn.Parameter(torch.full((d_k,), 1 / math.sqrt(d_k), device=device))
        self.k_weight = torch.nn.Parameter(torch.ones(d_k, device=device))
        if log_decay is None:
            log_decay = -torch.exp2(-torch.linspace(3, 8, n_heads))
        self.register_buffer("log_decay", log_decay.to(device=device, dtype=torch.float32))
        self.register_buffer("inv_freq", (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(device))
        self.register_buffer("axes", binding.rope_axes(sections, device or "cpu") if sections else None)

    def _qkv(self, x, positions):
        """x [B, T, d_model], positions [B, T] or [axes, B, T]: normalised and turned q, k, and v, [B, T, H, D] each."""
        B, T, _ = x.shape
        q, k = (t.view(B, T, self.H, self.Dk) for t in (x @ self.W_qk).split(self.H * self.Dk, -1))
        q, k = binding.qk_norm_rope(q, k, positions, self.inv_freq, self.axes, self.q_weight, self.k_weight, self.eps)
        return q, k, (x @ self.W_v).view(B, T, self.H, self.Dv)

    def forward(self, x, S0: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                cu_seqlens: Optional[torch.Tensor] = None, Tmax: Optional[int] = None):
        packed = cu_seqlens is not None
        if positions is None:
            if packed or self.axes is not None:
                raise ValueError("positions are needed with packed sequences and with several axes")
            positions = torch.arange(x.shape[1], dtype=torch.int32, device=x.device).expand(x.shape[:2]).contiguous()
        if not packed:
            q, k, v = self._qkv(x, positions)
            o, ST = binding.decay_linear_attention(q, k, v, self.log_decay, S0)
        else:
            q, k, v = self._qkv(x[None], positions.unsqueeze(-2))
            o, ST = binding.decay_linear_attention(q[0], k[0], v[0], self.log_decay, S0, cu_seqlens, Tmax)
        return o.flatten(-2) @ self.W_out, ST

    @torch.no_grad()
    def step(self, x, positions, S, slots: Optional[torch.Tensor] = None):
        """y [B, d_model] for one token of each request: x [B, d_model], positions [B] or [axes, B]; S [num_slots, H, Dk,
        Dv] fp32 is updated in place at ``slots`` (int32 [B]; negative: an idle row)."""
        q, k, v = self._qkv(x[:, None], positions.unsqueeze(-1))
        o = binding.gdn2_linear_decode_step(q[:, 0], k[:, 0], v[:, 0], self.log_decay, S, slots)
        return o.flatten(-2) @ self.W_out
