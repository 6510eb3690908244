"""Binding of further operators of a MoE layer's step (include/moe_step_ops.h).

Argument marshalling only, with the checks and the conventions of layer_ops.py.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional

import torch

from . import _check
from .layer_ops import _OpPlan, _tensor, _workspace

__all__ = ["GatePlan", "MoeLayerPlan", "QkNormRopePlan", "GradClipPlan", "SCORE_SOFTMAX", "SCORE_SIGMOID"]

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class GatePlan(_OpPlan):
    """The k experts of each of T tokens and their weights from router logits over
    E experts (C: moe_gate_plan / moe_gate_run), and the gradient of the weights
    (C: moe_gate_grad_run).  `score`: SCORE_SOFTMAX or SCORE_SIGMOID; `renormalize`:
    the weights of a token add to `scale`; `dtype`: of the logits, torch.float32 or
    torch.bfloat16."""

    def __init__(self, T: int, E: int, k: int, *, score: int = SCORE_SOFTMAX, renormalize: bool = True,
                 scale: float = 1.0, dtype=torch.float32, enable_pdl: bool = True, debug_checks: bool = False):
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, got {dtype}")
        self.T, self.E, self.k, self.score, self.dtype = int(T), int(E), int(k), int(score), dtype
        self._make("moe_gate_plan", self.T, self.E, self.k, self.score, int(bool(renormalize)), float(scale),
                   int(dtype is torch.bfloat16), enable_pdl=enable_pdl, debug_checks=debug_checks)

    def run(self, logits, expert_ids, topk_weights, bias=None, stream=None) -> None:
        """logits [T, E] -> expert_ids int32 and topk_weights FP32 [T, k]; bias FP32
        [E] (SCORE_SIGMOID) is added to the scores for the choice alone."""
        dev, pairs = self.device, (self.T, self.k)
        if bias is not None and self.score != SCORE_SIGMOID:
            raise ValueError("bias: only with SCORE_SIGMOID")
        _check(self._lib.moe_gate_run(
            self._h, _tensor("logits", logits, self.dtype, (self.T, self.E), dev),
            None if bias is None else _tensor("bias", bias, torch.float32, (self.E,), dev),
            _tensor("expert_ids", expert_ids, torch.int32, pairs, dev),
            _tensor("topk_weights", topk_weights, torch.float32, pairs, dev), self._stream(stream)), "moe_gate_run")

    def run_grad(self, d_topk_weights, logits, expert_ids, d_logits, stream=None) -> None:
        """d_topk_weights FP32 [T, k], run()'s logits and expert_ids -> d_logits [T, E]."""
        dev, pairs, rows = self.device, (self.T, self.k), (self.T, self.E)
        _check(self._lib.moe_gate_grad_run(
            self._h, _tensor("d_topk_weights", d_topk_weights, torch.float32, pairs, dev),
            _tensor("logits", logits, self.dtype, rows, dev), _tensor("expert_ids", expert_ids, torch.int32, pairs, dev),
            _tensor("d_logits", d_logits, self.dtype, rows, dev), self._stream(stream)), "moe_gate_grad_run")


class MoeLayerPlan(_OpPlan):
    """A whole MoE layer for a few tokens, T * k <= 4096: the gated experts of
    every token and their weighted sum (C: moe_small_layer_plan / _run).
    `dtype`: of x and the weights, torch.bfloat16 or torch.float8_e4m3fn (with
    FP32 scales per 128 columns of x and per 128 x 128 weights)."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, *, dtype=torch.bfloat16, enable_pdl: bool = True,
                 debug_checks: bool = False, sentinel_skip: bool = False):
        if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"dtype must be torch.bfloat16 or torch.float8_e4m3fn, got {dtype}")
        self.T, self.H, self.I, self.E, self.k, self.dtype = int(T), int(H), int(I), int(E), int(k), dtype
        self._make("moe_small_layer_plan", self.T, self.H, self.I, self.E, self.k, int(dtype is torch.float8_e4m3fn),
                   enable_pdl=enable_pdl, debug_checks=debug_checks, sentinel_skip=sentinel_skip)
        self._need = self.workspace_bytes()

    def set_wait_limit(self, limit_cycles: int) -> None:
        """SM cycles after which an on-chip wait of this plan's runs gives up and
        raises STATUS_TIMEOUT; 0: at once (C: moe_small_layer_set_wait_limit)."""
        _check(self._lib.moe_small_layer_set_wait_limit(self._h, int(limit_cycles)), "moe_small_layer_set_wait_limit")

    def run(self, x, expert_ids, topk_weights, w13, w2, out, workspace, x_sf=None, w13_sf=None, w2_sf=None,
            stream=None) -> None:
        """x [T, H], expert_ids int32 and topk_weights FP32 [T, k], w13 [E, 2 I, H]
        (gate rows, then up rows), w2 [E, H, I] -> out bf16 [T, H]; for E4M3 with
        x_sf [T, ceil(H/128)], w13_sf [E, 2 I / 128, ceil(H/128)], w2_sf [E, ceil(H/128), I / 128]."""
        f32, dev, dt = torch.float32, self.device, self.dtype
        T, H, I, E, pairs = self.T, self.H, self.I, self.E, (self.T, self.k)
        sf = [None, None, None]
        if dt is torch.float8_e4m3fn:
            hb, ib = -(-H // 128), I // 128
            sf = [_tensor("x_sf", x_sf, f32, (T, hb), dev), _tensor("w13_sf", w13_sf, f32, (E, 2 * ib, hb), dev),
                  _tensor("w2_sf", w2_sf, f32, (E, hb, ib), dev)]
        elif x_sf is not None or w13_sf is not None or w2_sf is not None:
            raise ValueError("x_sf, w13_sf, w2_sf: this plan was made for bf16")
        ws, ws_bytes = _workspace(workspace, self._need, dev)
        _check(self._lib.moe_small_layer_run(
            self._h, _tensor("x", x, dt, (T, H), dev), sf[0], _tensor("expert_ids", expert_ids, torch.int32, pairs, dev),
            _tensor("topk_weights", topk_weights, f32, pairs, dev), _tensor("w13", w13, dt, (E, 2 * I, H), dev), sf[1],
            _tensor("w2", w2, dt, (E, H, I), dev), sf[2], _tensor("out", out, torch.bfloat16, (T, H), dev), ws, ws_bytes,
            self._stream(stream)), "moe_small_layer_run")


_HEADS = 24        # bytes of a moe_heads_t: address, token stride, head stride, 64 bits each


class QkNormRopePlan(_OpPlan):
    """RMSNorm of every query and key head of T tokens with the position rotation
    in the same pass (C: moe_qk_norm_rope_plan / _run), and its gradient (C:
    moe_qk_norm_rope_grad_run, which takes the workspace).  `rotary_dim`: elements
    of a head that turn (default: all D); `interleaved`: pairs (2 i, 2 i + 1) instead
    of (i, i + rotary_dim / 2); `dtype`: torch.bfloat16 or torch.float16."""

    def __init__(self, T: int, heads_q: int, heads_k: int, D: int, *, rotary_dim: Optional[int] = None,
                 interleaved: bool = False, dtype=torch.bfloat16, max_positions: int, enable_pdl: bool = True,
                 debug_checks: bool = False):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        self.T, self.heads_q, self.heads_k, self.D, self.dtype = int(T), int(heads_q), int(heads_k), int(D), dtype
        self.rotary_dim, self.max_positions = self.D if rotary_dim is None else int(rotary_dim), int(max_positions)
        self._make("moe_qk_norm_rope_plan", self.T, self.heads_q, self.heads_k, self.D, self.rotary_dim,
                   int(bool(interleaved)), int(dtype is torch.float16), self.max_positions, enable_pdl=enable_pdl,
                   debug_checks=debug_checks)
        self._need = self.workspace_bytes()

    def _heads(self, name: str, t, heads: int) -> tuple:
        shape = (self.T, heads, self.D)
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if t.dtype is not self.dtype or t.shape != shape:
            raise ValueError(f"{name}: expected {self.dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on the plan's device {self.device}, not on {t.device}")
        token, head, one = t.stride()
        if one != 1 or token < 0 or head < 0:
            raise ValueError(f"{name}: the elements of a head must lie together, got strides {t.stride()}")
        # the stride of a dimension of one is never taken
        return t.data_ptr(), token if self.T > 1 else 0, head if heads > 1 else 0

    def _shared(self, gamma_q, gamma_k, cos_sin, positions):
        dt, dev, D = self.dtype, self.device, (self.D,)
        return (_tensor("gamma_q", gamma_q, dt, D, dev), _tensor("gamma_k", gamma_k, dt, D, dev),
                _tensor("cos_sin", cos_sin, torch.float32, (self.max_positions, self.rotary_dim), dev),
                _tensor("positions", positions, torch.int32, (self.T,), dev))

    def run(self, q, k, gamma_q, gamma_k, eps: float, cos_sin, positions, q_out, k_out, stream=None) -> None:
        """q [T, heads_q, D] and k [T, heads_k, D], strided (parts of a packed tensor),
        gammas [D], cos_sin FP32 [max_positions, rotary_dim] (cosines, then sines),
        positions int32 [T] -> q_out, k_out (may be q and k)."""
        gq, gk, table, pos = self._shared(gamma_q, gamma_k, cos_sin, positions)
        hq, hk = self.heads_q, self.heads_k
        heads = array("q", (*self._heads("q", q, hq), *self._heads("k", k, hk), *self._heads("q_out", q_out, hq),
                            *self._heads("k_out", k_out, hk)))
        at = heads.buffer_info()[0]
        _check(self._lib.moe_qk_norm_rope_run(self._h, at, at + _HEADS, gq, gk, eps, table, pos, at + 2 * _HEADS,
                                              at + 3 * _HEADS, self._stream(stream)), "moe_qk_norm_rope_run")

    def run_grad(self, d_q_out, d_k_out, q, k, gamma_q, gamma_k, eps: float, cos_sin, positions, d_q, d_k, d_gamma_q,
                 d_gamma_k, workspace, stream=None) -> None:
        """d_q_out, d_k_out and run()'s inputs -> d_q, d_k (strided as well; may be
        d_q_out and d_k_out) and d_gamma_q, d_gamma_k FP32 [D]."""
        f32, dev = torch.float32, self.device
        gq, gk, table, pos = self._shared(gamma_q, gamma_k, cos_sin, positions)
        ws, ws_bytes = _workspace(workspace, self._need, dev)
        hq, hk = self.heads_q, self.heads_k
        heads = array("q", (*self._heads("d_q_out", d_q_out, hq), *self._heads("d_k_out", d_k_out, hk), *self._heads("q", q, hq),
                            *self._heads("k", k, hk), *self._heads("d_q", d_q, hq), *self._heads("d_k", d_k, hk)))
        at = heads.buffer_info()[0]
        _check(self._lib.moe_qk_norm_rope_grad_run(
            self._h, at, at + _HEADS, at + 2 * _HEADS, at + 3 * _HEADS, gq, gk, eps, table, pos, at + 4 * _HEADS,
            at + 5 * _HEADS, _tensor("d_gamma_q", d_gamma_q, f32, (self.D,), dev),
            _tensor("d_gamma_k", d_gamma_k, f32, (self.D,), dev), ws, ws_bytes, self._stream(stream)), "moe_qk_norm_rope_grad_run")


_GRAD_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class GradClipPlan(_OpPlan):
    """The L2 norm of many tensors together, and the tensors scaled to a largest
    norm (C: moe_grad_clip_plan / _run).  `numels`: elements of each; `dtypes`: their
    types (torch.float32, torch.bfloat16, torch.float16), or one for all."""

    def __init__(self, numels, dtypes=torch.float32, *, enable_pdl: bool = True, debug_checks: bool = False):
        self.numels = [int(n) for n in numels]
        self.dtypes = [dtypes] * len(self.numels) if isinstance(dtypes, torch.dtype) else list(dtypes)
        if len(self.dtypes) != len(self.numels):
            raise ValueError(f"dtypes: expected one or {len(self.numels)}, got {len(self.dtypes)}")
        for d in self.dtypes:
            if d not in _GRAD_TYPES:
                raise ValueError(f"dtypes: torch.float32, torch.bfloat16 or torch.float16, got {d}")
        n = len(self.numels)
        self._make("moe_grad_clip_plan", n, (ctypes.c_int64 * n)(*self.numels),
                   (ctypes.c_int * n)(*[_GRAD_TYPES[d] for d in self.dtypes]), enable_pdl=enable_pdl,
                   debug_checks=debug_checks)
        self._need = self.workspace_bytes()

    def _addresses(self, name: str, tensors) -> array:
        if len(tensors) != len(self.numels):
            raise ValueError(f"{name}: expected {len(self.numels)} tensors, got {len(tensors)}")
        T, dev = torch.Tensor, self.device
        try:        # all at once: a quarter of the time of looking at them one by one
            if list(map(T.numel, tensors)) == self.numels and [t.dtype for t in tensors] == self.dtypes and \
                    all(map(T.is_contiguous, tensors)) and {*map(T.get_device, tensors)} <= {-1 if dev.index is None else dev.index}:
                return array("Q", map(T.data_ptr, tensors))
        except TypeError:
            pass    # one of them is no tensor
        for i, (t, n, dt) in enumerate(zip(tensors, self.numels, self.dtypes)):
            if not isinstance(t, T) or t.dtype is not dt or t.numel() != n:
                raise ValueError(f"{name}[{i}]: expected a tensor of {n} elements of {dt}")
            if not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{name}[{i}] must be contiguous and on the plan's device {dev}")
        raise ValueError(f"{name}: not the plan's tensors")

    def run(self, grads, max_norm: float, norm, workspace, out=None, *, eps: float = 1e-6, stream=None) -> None:
        """norm FP32 [1] = the norm of all grads together; out[i] (default: grads[i], in
        place) = grads[i] * min(1, max_norm / (norm + eps)).  A norm that is not finite scales nothing."""
        dev = self.device
        src = self._addresses("grads", grads)
        dst = src if out is None else self._addresses("out", out)
        ws, ws_bytes = _workspace(workspace, self._need, dev)
        _check(self._lib.moe_grad_clip_run(self._h, src.buffer_info()[0], dst.buffer_info()[0], max_norm, eps,
                                           _tensor("norm", norm, torch.float32, (1,), dev), ws, ws_bytes,
                                           self._stream(stream)), "moe_grad_clip_run")
