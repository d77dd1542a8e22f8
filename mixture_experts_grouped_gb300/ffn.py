"""Serving-side feed-forward pieces around the expert layer.

:class:`FewTokensLayer` is the expert layer for at most 32 tokens (buffers and
one call); :class:`SharedExpert` a dense SwiGLU expert on E4M3 weights with
block scales; :class:`FeedForward` the feed-forward half of a decoder layer
from them: residual addition and norm, the routed experts, the shared expert
added to them. As in :mod:`layer`, PyTorch only provides device memory and the
stream, every step runs in libmoe.so, nothing synchronises with the host, and
buffers are allocated once.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import layer as L
from . import moe as M


class FewTokensLayer:
    """Buffers for the whole expert layer at one (T, H, I, E, k) shape, T <= 32, and its one call."""

    def __init__(self, T, H, I, E, k, act, w_gate_up: L.DeviceWeight, w_down: L.DeviceWeight, device="cuda",
                 renormalize: bool = True):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.act, self.act_code = act, M.ACT_CODES[act]
        self.w_gate_up, self.w_down, self.renormalize = w_gate_up, w_down, renormalize
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws_bytes = M.moe_few_tokens_workspace_size(T, k, I)
        self.ws = torch.empty(max(1, self.ws_bytes), dtype=torch.uint8, device=device)
        self.out = torch.empty((T, H), dtype=L.act_dtype(act), device=device)

    @staticmethod
    def takes(T, H, I, E, k, w_gate_up: L.DeviceWeight, w_down: L.DeviceWeight) -> bool:
        """Whether the call takes a layer that the grouped path takes too: few tokens, weights
        of one format, and sizes that its row numbers hold."""
        pairs = T * k
        return (T <= M.MOE_MAX_FEW_TOKENS and w_gate_up.desc.format == w_down.desc.format and 2 * I * H < 2 ** 30
                and (min(E, pairs) + pairs // 8) * I < 2 ** 31)

    def forward(self, x, logits=None, stream=None):
        """The layer on x [T, H]; returns its output buffer. Without logits the
        routing already in ``topk_ids`` / ``topk_weights`` is used."""
        M.moe_few_tokens(x, self.act_code, logits, self.topk_ids, self.topk_weights, self.w_gate_up.desc,
                         self.w_down.desc, self.T, self.k, self.H, self.I, self.E, self.renormalize, self.out,
                         self.err, self.ws, self.ws_bytes, stream)
        return self.out


def quant_buffers(rows: int, cols: int, device):
    """Codes and scales of a quantised [rows, cols] tensor."""
    g = -(-cols // M.MOE_QUANT_GROUP)
    return (torch.empty((rows, cols), dtype=torch.uint8, device=device),
            torch.empty((rows, g), dtype=torch.float32, device=device))


def _require_shape(what: str, t: torch.Tensor, *shape: int) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")


@dataclass
class BlockFp8Weight:
    """E4M3 codes uint8 [N, K] with f32 scales [ceil(N / 128), ceil(K / 128)]."""
    codes: torch.Tensor
    scales: torch.Tensor

    def require(self, what: str, n: int, k: int) -> None:
        g = M.MOE_QUANT_GROUP
        _require_shape(f"{what} weight", self.codes, n, k)
        _require_shape(f"scales of the {what} weight", self.scales, -(-n // g), -(-k // g))


class SharedExpert:
    """A dense SwiGLU expert on block-scaled E4M3 weights: gate/up product,
    SiLU-mul, down product, optionally added to another output."""

    def __init__(self, T, H, I, act, w_gate_up: BlockFp8Weight, w_down: BlockFp8Weight, device="cuda"):
        w_gate_up.require("gate/up", 2 * I, H)
        w_down.require("down", H, I)
        self.T, self.H, self.I = T, H, I
        self.act_code = M.ACT_CODES[act]
        self.w_gate_up, self.w_down = w_gate_up, w_down
        dt = L.act_dtype(act)
        self.gate_up = torch.empty((T, 2 * I), dtype=dt, device=device)
        self.q, self.q_scales = quant_buffers(T, I, device)
        self.out = torch.empty((T, H), dtype=dt, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def forward(self, xq, xq_scales, addend=None, stream=None):
        """The expert on quantised rows [T, H], plus ``addend`` [T, H]; returns its output buffer."""
        M.moe_block_fp8_gemm(xq, xq_scales, self.w_gate_up.codes, self.w_gate_up.scales, None, self.gate_up,
                             self.act_code, self.T, 2 * self.I, self.H, self.err, stream)
        M.moe_silu_mul_quant(self.gate_up, self.act_code, self.T, self.I, self.q, self.q_scales, stream)
        M.moe_block_fp8_gemm(self.q, self.q_scales, self.w_down.codes, self.w_down.scales, addend, self.out,
                             self.act_code, self.T, self.H, self.I, self.err, stream)
        return self.out


_WEIGHT_BITS = {M.MOE_W_BF16: 16.0, M.MOE_W_GPTQ_INT4: 4.15, M.MOE_W_NVFP4: 4.5, M.MOE_W_FP8_E4M3: 8.0}


def few_tokens_pay(fmt: int, T: int, H: int, I: int, E: int, k: int) -> bool:
    """Whether the few-token call beats the grouped path on a layer that it takes.

    It saves the grouped path's five launches and its sort, about 20 us; the grouped GEMMs
    read weights of experts with several tokens faster. So the grouped path pays where the
    touched weights are many and an expert has many tokens (us, few-token call / grouped):
    bf16, 8 experts of 4096 x 14336, k = 2: 127 / 134 at T = 1, 214 / 207 at 2, 479 / 435 at
    16, 754 / 438 at 32; 16 of 4096 x 2048, k = 4: 148 / 146 at T = 12, 165 / 147 at 24; 32
    of 2048 x 768, k = 8: 70 / 82 at 24, 89 / 83 at 32. FP8, the first layer: 276 / 298 at 16,
    301 / 299 at 24, 332 / 299 at 32; the second 113 / 116 at 32. GPTQ, the first: 230 / 235
    at 16, 255 / 236 at 24, 335 / 236 at 32; the second 86 / 93 at 16, 97 / 94 at 24, 119 / 94
    at 32; the third 57 / 62 at 32. NVFP4, the first 327 / 339 at 32."""
    per_expert = T * k / E
    touched = E * (1.0 - (1.0 - k / E) ** T) * 3 * H * I * _WEIGHT_BITS.get(fmt, 16.0) / 8  # bytes, expected
    if fmt == M.MOE_W_BF16:
        return touched < 1.1e9 and per_expert * touched < 2.3e9
    if fmt == M.MOE_W_GPTQ_INT4:
        return per_expert < 6 or per_expert * touched < 1.0e9
    return per_expert * touched < 6.8e9


class FeedForward:
    """The feed-forward half of a decoder layer at one shape:

        r = x + residual,  y = norm(r),  out = experts(y) + shared(e4m3(y))

    ``forward`` returns (out, r), what the next layer takes. The routed experts
    run as :class:`FewTokensLayer` where that takes them (up to 32 tokens,
    weights of one format) and is faster (:func:`few_tokens_pay`), and as
    :class:`layer.MoeLayer` elsewhere; the router weight is f32 [H, E]. A shared
    expert of another T, H or activation type is refused (ValueError). There is
    no LoRA here: a layer with adapters runs :class:`layer.MoeLayer`'s steps.
    """

    def __init__(self, T, H, I, E, k, act, norm_weight, w_router, w_gate_up: L.DeviceWeight, w_down: L.DeviceWeight,
                 shared: Optional[SharedExpert] = None, eps: float = 1e-6, bs: int = 16, device="cuda",
                 renormalize: bool = True):
        self.T, self.H, self.E, self.k, self.eps, self.renormalize = T, H, E, k, eps, renormalize
        self.act_code = M.ACT_CODES[act]
        _require_shape("norm_weight", norm_weight, H)
        _require_shape("w_router", w_router, H, E)
        if shared is not None and (shared.T, shared.H, shared.act_code) != (T, H, self.act_code):
            raise ValueError(f"the shared expert is one of T={shared.T}, H={shared.H}, activation type "
                             f"{shared.act_code}, the block of T={T}, H={H}, {self.act_code}")
        self.norm_weight, self.w_router, self.shared = norm_weight, w_router, shared
        dt = L.act_dtype(act)
        self.residual = torch.empty((T, H), dtype=dt, device=device)
        self.y = torch.empty((T, H), dtype=dt, device=device)
        self.q, self.q_scales = quant_buffers(T, H, device) if shared is not None else (None, None)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=device)
        if (FewTokensLayer.takes(T, H, I, E, k, w_gate_up, w_down)
                and few_tokens_pay(w_gate_up.desc.format, T, H, I, E, k)):
            self.experts = FewTokensLayer(T, H, I, E, k, act, w_gate_up, w_down, device, renormalize)
        else:
            self.experts = L.MoeLayer(T, H, I, E, k, bs, act, w_gate_up, w_down, device, renormalize=renormalize)

    def forward(self, x, residual=None, stream=None):
        M.moe_add_rmsnorm_quant(x, residual, self.act_code, self.norm_weight, self.eps, self.T, self.H, self.residual,
                                self.y, self.q, self.q_scales, stream)
        ex = self.experts
        M.moe_router_topk_softmax(self.y, self.act_code, self.w_router, self.T, self.H, self.E, self.k,
                                  self.renormalize, self.logits, ex.topk_ids, ex.topk_weights, stream)
        if isinstance(ex, FewTokensLayer):
            out = ex.forward(self.y, None, stream)
        else:
            ex.align(stream)
            ex.gate_up(self.y, stream)
            ex.down(stream)
            ex.combine(stream)
            out = ex.out
        if self.shared is not None:
            out = self.shared.forward(self.q, self.q_scales, out, stream)
        return out, self.residual
