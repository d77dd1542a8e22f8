"""Training steps of the expert layer and of a dense block.

:class:`MoeTrainLayer` is the expert layer with its gradients, on ragged spans
(no padding); :class:`DenseMlp` two dense products with biases, an activation
between them and a residual, with theirs. As in :mod:`layer`, PyTorch only
provides device memory and the stream, every step runs in libmoe.so, nothing
synchronises with the host and buffers are allocated once, so a forward and a
backward pass can be captured in a CUDA graph. There is no autograd here:
``backward`` is called with the output's gradient and writes the gradients
into buffers of the object. Weights and inputs are on the object's device, and a
pass runs while that is the current one; anything else is refused (ValueError).
"""

from __future__ import annotations

import torch

from . import layer as L
from . import moe as M
from .ffn import _Buffers, _cuda_device, _require, _require_current


class MoeTrainLayer:
    """Buffers of one (T, H, I, E, k) shape, a forward and a backward pass:

        out[t] = sum_j w_tj swiglu(x[t] Wg_e^T) Wd_e^T,   e, w = routing of logits[t]

    Weights are 16-bit tensors of the activation type, ``w_gate_up`` [E, 2 I, H]
    (gate rows first) and ``w_down`` [E, H, I]; their gradients ``d_gate_up`` and
    ``d_down`` are f32, zeros at first. ``backward`` uses what the last ``forward`` left
    in the buffers, and its logits. It may be called several times for one forward
    pass. An object runs one pass at a time: calls on several streams share its buffers."""

    def __init__(self, T, H, I, E, k, act, w_gate_up: torch.Tensor, w_down: torch.Tensor, device="cuda",
                 renormalize: bool = True):
        dt = self.dtype = L.act_dtype(act)
        if T < 1:
            raise ValueError(f"T={T}: a step needs a token")
        device = self.device = _cuda_device(device)
        _require("w_gate_up", w_gate_up, device, dt, E, 2 * I, H)
        _require("w_down", w_down, device, dt, E, H, I)
        self.T, self.H, self.I, self.E, self.k, self.P = T, H, I, E, k, T * k
        self.act_code, self.renormalize = M.ACT_CODES[act], renormalize
        self.w_gate_up, self.w_down = w_gate_up, w_down
        P = self.P

        def i32(n):
            return torch.empty(max(1, n), dtype=torch.int32, device=device)

        def rows(n, cols):
            return torch.empty((n, cols), dtype=dt, device=device)

        def f32(*shape):
            return torch.empty(shape, dtype=torch.float32, device=device)

        # block_size 1: spans without padding, max_padded = P
        self.topk_ids, self.topk_weights = torch.empty((T, k), dtype=torch.int32, device=device), f32(T, k)
        self.sorted_token_ids, self.expert_ids, self.pair_to_row = i32(P), i32(P), i32(P)
        self.offsets, self.total = i32(E + 1), i32(1)
        self.align_ws_bytes = M.moe_align_workspace_size(P, E)
        self.align_ws = torch.empty(max(1, self.align_ws_bytes), dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.ones = torch.ones((T, k), dtype=torch.float32, device=device)
        self.xs, self.gate_up, self.h, self.y = rows(P, H), rows(P, 2 * I), rows(P, I), rows(P, H)
        self.out = rows(T, H)
        self.d_y, self.d_h, self.d_gu, self.d_xs, self.d_x = rows(P, H), rows(P, I), rows(P, 2 * I), rows(P, H), rows(T, H)
        self.d_weights, self.d_logits = f32(T, k), f32(T, E)
        self.d_gate_up, self.d_down = f32(E, 2 * I, H).zero_(), f32(E, H, I).zero_()
        self.logits = None
        self._own = _Buffers(self, "topk_ids", "topk_weights", "sorted_token_ids", "expert_ids", "pair_to_row", "offsets",
                             "total", "align_ws", "err", "ones", "xs", "gate_up", "h", "y", "out", "d_y", "d_h", "d_gu",
                             "d_xs", "d_x", "d_weights", "d_logits", "d_gate_up", "d_down")
        self._before_x = ("topk_ids", "topk_weights", "sorted_token_ids", "expert_ids", "pair_to_row", "offsets", "total",
                          "align_ws", "err", "xs")  # written before x has been read, or while it is

    def forward(self, x, logits, stream=None):
        """The layer on x [T, H] routed by logits [T, E]; returns its output buffer. logits is kept for ``backward``, must
        not change before it and is no buffer of the layer; x may be one that the pass has read by the time it writes
        it, like an earlier output."""
        T, H, I, E, k, P, act = self.T, self.H, self.I, self.E, self.k, self.P, self.act_code
        _require_current(self.device)
        _require("x", x, self.device, self.dtype, T, H)
        _require("logits", logits, self.device, torch.float32, T, E)
        self._own.refuse("x", x, self._before_x)
        self._own.refuse("logits", logits)
        self.logits = None  # (until the pass is complete: a call of it may be refused)
        M.moe_route_topk_softmax(logits, self.topk_ids, self.topk_weights, T, E, k, self.renormalize, stream)
        M.moe_align_block_size(self.topk_ids, P, E, 1, P, self.sorted_token_ids, self.expert_ids, self.offsets,
                               self.total, self.pair_to_row, self.err, self.align_ws, self.align_ws_bytes, stream)
        M.moe_dispatch(x, act, self.pair_to_row, self.xs, T, H, k, P, self.err, stream)
        M.moe_ragged_gemm(self.xs, act, self.w_gate_up, False, self.offsets, P, 2 * I, H, E, self.gate_up, self.err,
                          stream)
        M.moe_swiglu(self.gate_up, act, P, I, self.h, stream)
        M.moe_ragged_gemm(self.h, act, self.w_down, False, self.offsets, P, H, I, E, self.y, self.err, stream)
        M.moe_combine(self.y, act, self.pair_to_row, self.topk_weights, self.out, T, H, k, P, self.err, stream)
        self.logits = logits
        return self.out

    def backward(self, d_out, accumulate: bool = False, stream=None):
        """Gradients of the last forward pass from its output's, d_out [T, H]: returns (d_x, d_logits);
        the weights' are in ``d_gate_up`` and ``d_down``, added to what is there if ``accumulate``."""
        T, H, I, E, k, P, act = self.T, self.H, self.I, self.E, self.k, self.P, self.act_code
        if self.logits is None:
            raise RuntimeError("backward without a forward pass")
        _require_current(self.device)
        _require("d_out", d_out, self.device, self.dtype, T, H)
        self._own.refuse("d_out", d_out, ("d_y", "d_weights", "err"))
        M.moe_combine_backward(d_out, self.y, act, self.pair_to_row, self.topk_weights, self.d_y, self.d_weights, T, H,
                               k, P, self.err, stream)
        M.moe_ragged_gemm(self.d_y, act, self.w_down, True, self.offsets, P, H, I, E, self.d_h, self.err, stream)
        M.moe_ragged_wgrad(self.d_y, self.h, act, self.offsets, P, H, I, E, self.d_down if accumulate else None,
                           self.d_down, True, self.err, stream)
        M.moe_swiglu_backward(self.gate_up, self.d_h, act, P, I, self.d_gu, None, stream)
        M.moe_ragged_gemm(self.d_gu, act, self.w_gate_up, True, self.offsets, P, 2 * I, H, E, self.d_xs, self.err,
                          stream)
        M.moe_ragged_wgrad(self.d_gu, self.xs, act, self.offsets, P, 2 * I, H, E,
                           self.d_gate_up if accumulate else None, self.d_gate_up, True, self.err, stream)
        M.moe_combine(self.d_xs, act, self.pair_to_row, self.ones, self.d_x, T, H, k, P, self.err, stream)
        M.moe_route_backward(self.logits, self.topk_ids, self.topk_weights, self.d_weights, self.d_logits, T, E, k,
                             self.renormalize, self.err, stream)
        return self.d_x, self.d_logits


class DenseMlp:
    """A dense block at one (T, H, I) shape, forward and backward:

        out = f(x w1^T + b1) w2^T + b2 (+ residual)

    ``w1`` [I, H], ``w2`` [H, I] and the biases (or None) are 16-bit tensors of the
    activation type, ``fn`` a name of ``moe.FN_CODES``. The weights' gradients
    ``d_w1`` and ``d_w2`` and the biases' ``d_b1`` and ``d_b2`` are f32, zeros at first;
    the residual's is the output's. An object runs one pass at a time."""

    def __init__(self, T, H, I, act, fn, w1, b1, w2, b2, device="cuda"):
        dt = self.dtype = L.act_dtype(act)
        if T < 1:
            raise ValueError(f"T={T}: a step needs a token")
        device = self.device = _cuda_device(device)
        for name, t, shape in (("w1", w1, (I, H)), ("w2", w2, (H, I)), ("b1", b1, (I,)), ("b2", b2, (H,))):
            if t is not None:
                _require(name, t, device, dt, *shape)
        self.T, self.H, self.I = T, H, I
        self.act_code, self.fn = M.ACT_CODES[act], M.FN_CODES[fn]
        self.w1, self.b1, self.w2, self.b2 = w1, b1, w2, b2

        def rows(cols):
            return torch.empty((T, cols), dtype=dt, device=device)

        def f32(*shape):
            return torch.empty(shape, dtype=torch.float32, device=device)

        self.pre, self.h, self.out, self.d_h, self.d_x = rows(I), rows(I), rows(H), rows(I), rows(H)
        self.d_w1, self.d_w2 = f32(I, H).zero_(), f32(H, I).zero_()
        self.d_b1 = f32(I).zero_() if b1 is not None else None
        self.d_b2 = f32(H).zero_() if b2 is not None else None
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.x = None
        self._own = _Buffers(self, "pre", "h", "out", "d_h", "d_x", "d_w1", "d_w2", "d_b1", "d_b2", "err")

    def forward(self, x, residual=None, stream=None):
        """The block on x [T, H]; returns its output buffer. x is kept for ``backward``, must not change before it
        and is no buffer of the block; the residual may be the output buffer itself."""
        _require_current(self.device)
        _require("x", x, self.device, self.dtype, self.T, self.H)
        self._own.refuse("x", x)
        if residual is not None:
            _require("residual", residual, self.device, self.dtype, self.T, self.H)
            self._own.refuse("residual", residual, ("pre", "h", "out", "err"), in_place="out")
        self.x = None  # (until the pass is complete)
        M.moe_dense_gemm(x, self.act_code, self.w1, self.b1, self.fn, None, self.pre, self.h, self.T, self.I, self.H,
                         self.err, stream)
        M.moe_dense_gemm(self.h, self.act_code, self.w2, self.b2, M.MOE_FN_NONE, residual, None, self.out, self.T,
                         self.H, self.I, self.err, stream)
        self.x = x
        return self.out

    def backward(self, d_out, accumulate: bool = False, stream=None):
        """Gradients of the last forward pass from its output's, d_out [T, H]: returns d_x; the weights'
        and biases' are in ``d_w1`` .. ``d_b2``, added to what is there if ``accumulate``."""
        T, H, I, act = self.T, self.H, self.I, self.act_code
        if self.x is None:
            raise RuntimeError("backward without a forward pass")
        _require_current(self.device)
        _require("d_out", d_out, self.device, self.dtype, T, H)
        self._own.refuse("d_out", d_out, ("d_b2", "d_w2", "d_h", "err"))
        if self.d_b2 is not None:
            M.moe_bias_act_backward(d_out, None, act, M.MOE_FN_NONE, T, H, None, self.d_b2, accumulate,
                                    stream)
        M.moe_ragged_wgrad(d_out, self.h, act, None, T, H, I, 1, self.d_w2 if accumulate else None, self.d_w2, True,
                           self.err, stream)
        M.moe_ragged_gemm(d_out, act, self.w2, True, None, T, H, I, 1, self.d_h, self.err, stream)
        if self.fn != M.MOE_FN_NONE or self.d_b1 is not None:
            M.moe_bias_act_backward(self.d_h, self.pre, act, self.fn, T, I, self.d_h, self.d_b1,
                                    accumulate, stream)
        M.moe_ragged_wgrad(self.d_h, self.x, act, None, T, I, H, 1, self.d_w1 if accumulate else None, self.d_w1, True,
                           self.err, stream)
        M.moe_ragged_gemm(self.d_h, act, self.w1, True, None, T, I, H, 1, self.d_x, self.err, stream)
        return self.d_x
