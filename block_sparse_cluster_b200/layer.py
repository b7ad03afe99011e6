"""A transformer layer's attention around the decoupled sparse attention step, in 8-bit weights.

``DecoupledLayer`` takes hidden states instead of Q, K and V: it adds them to the residual stream,
norms them (a root-mean-square norm of fixed weight: no shift, no scale per sample, no gate),
projects them with 8-bit integer products, turns queries and keys by their rotary positions, runs
Reassign Cache and the decoupled attention, and projects the output back.  Every step is one call
of the library's operators; this module owns the buffers between them.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import (DAError, DecoupledAttention, Dims, Rope, da_linear_i8, da_quantize_i8, da_rms_norm_i8, da_rope)


def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


def _codes(rows: int, width: int, device) -> torch.Tensor:
    """[rows, width] int8 whose rows start on 16 bytes, which the products read fastest."""
    return torch.zeros(rows, _pad16(width), dtype=torch.int8, device=device)[:, :width]


def quantize_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of a weight [channels, width] (bf16 or fp32, on the GPU), a scale per channel."""
    q = _codes(w.shape[0], w.shape[1], w.device)
    scale = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
    return da_quantize_i8(w, q, scale)


@dataclass
class LayerWeights:
    """Weights of one layer: codes [channels, width] int8 with a scale per channel.  Queries and
    keys are one product, values one, the output one.  Norm weights are of the layer's dtype, biases fp32."""
    norm: Optional[torch.Tensor]              # [width]
    qk: Tuple[torch.Tensor, torch.Tensor]     # codes [2*H*d, width] (queries first), scales
    v: Tuple[torch.Tensor, torch.Tensor]      # codes [H*d, width], scales
    out: Tuple[torch.Tensor, torch.Tensor]    # codes [width, H*d], scales
    q_norm: Optional[torch.Tensor] = None     # [d] (a head) or [H*d] (all heads)
    k_norm: Optional[torch.Tensor] = None
    qk_bias: Optional[torch.Tensor] = None
    v_bias: Optional[torch.Tensor] = None
    out_bias: Optional[torch.Tensor] = None

    @staticmethod
    def quantize(norm, wq, wk, wv, wo, **rest) -> "LayerWeights":
        """From weights [channels, width] in bf16 or fp32 on the GPU; `rest`: the optional fields."""
        return LayerWeights(norm, quantize_weight(torch.cat([wq, wk])), quantize_weight(wv), quantize_weight(wo), **rest)


class DecoupledLayer:
    """Buffers of one layer shape plus the two halves of its step, ``project`` and ``attend``.

    The attention engine is ``engine`` (its plan is prepared once with ``prepare``); Q, K and V of
    the last ``project`` are ``Q``, ``K`` and ``V`` [B,H,N,d], for the initial clustering of the keys.
    Every call makes the layer's device current, whose current stream is the default one.
    """

    def __init__(self, dims: Dims, width: int, weights: LayerWeights, rope: Rope, eps: float = 1e-6, device="cuda"):
        self.dims, self.width, self.weights, self.rope, self.eps = dims, width, weights, rope, eps
        B, H, N, d = dims.B, dims.H, dims.N, dims.d
        tokens, channels = B * N, H * d
        for name, (codes, scales), shape in (("qk", weights.qk, (2 * channels, width)), ("v", weights.v, (channels, width)),
                                             ("out", weights.out, (width, channels))):
            if tuple(codes.shape) != shape or tuple(scales.shape) != shape[:1]:
                raise DAError(2, f"DecoupledLayer: weight {name} has to be {list(shape)}")
        self.engine = DecoupledAttention(dims, device)
        f32, like = dict(dtype=torch.float32, device=device), dict(dtype=dims.dtype, device=device)
        self._x, self._x_scale = _codes(tokens, width, device), torch.empty(tokens, **f32)
        self._o, self._o_scale = _codes(tokens, channels, device), torch.empty(tokens, **f32)
        self._qk = torch.empty(tokens, 2 * channels, **like)
        self.Q, self.K, self.V, self.O = (torch.empty(B, H, N, d, **like) for _ in range(4))

    def _on_device(self):
        # the attention's calls run on the current device, unlike the layer operators, which run on their tensors'
        return torch.cuda.device(self.Q.device)

    def prepare(self, kv_idx: torch.Tensor, kv_cnt: torch.Tensor, stream=None):
        with self._on_device():
            return self.engine.prepare(kv_idx, kv_cnt, stream)

    def project(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, stream=None) -> None:
        """Hidden states x [B, N, width] to Q, K and V.  With a residual stream [B, N, width], which
        becomes residual + x in place, the norm is of the sum."""
        w, (B, H, N, d) = self.weights, self.Q.shape
        rows = x.view(B * N, self.width)
        total = None if residual is None else residual.view(B * N, self.width)
        with self._on_device():
            da_rms_norm_i8(rows, w.norm, self._x, self._x_scale, residual=total, sum_out=total, eps=self.eps, stream=stream)
            ws = self.engine.ws
            da_linear_i8(self._x, self._x_scale, *w.qk, self._qk, ws, bias=w.qk_bias, stream=stream)
            da_linear_i8(self._x, self._x_scale, *w.v, self.V, ws, bias=w.v_bias, stream=stream)
            slots = self._qk.view(B, N, 2, H, d)
            for slot, norm, out in ((0, w.q_norm, self.Q), (1, w.k_norm, self.K)):
                da_rope(slots[:, :, slot].permute(0, 2, 1, 3), out, self.rope, weight=norm, eps=self.eps, stream=stream)

    def attend(self, centroids: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
        """Attention of the projected Q, K and V, and its projection into out [B, N, width]."""
        w, (B, H, N, d) = self.weights, self.Q.shape
        with self._on_device():
            self.engine.step(self.Q, self.K, self.V, centroids, self.O, stream=stream)
            da_quantize_i8(self.O, self._o, self._o_scale, stream=stream)
            da_linear_i8(self._o, self._o_scale, *w.out, out.view(B * N, self.width), self.engine.ws, bias=w.out_bias,
                         stream=stream)
        return out

    def step(self, x: torch.Tensor, centroids: torch.Tensor, out: torch.Tensor,
             residual: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        self.project(x, residual, stream)
        return self.attend(centroids, out, stream)

    def status(self, stream=None) -> int:
        with self._on_device():
            return self.engine.status(stream)
