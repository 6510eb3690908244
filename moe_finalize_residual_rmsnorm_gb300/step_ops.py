"""Binding of further operators of a MoE layer's step (include/moe_step_ops.h).

Argument marshalling only, with the checks and the conventions of layer_ops.py.
"""
from __future__ import annotations

import torch

from . import _check
from .layer_ops import _OpPlan, _tensor, _workspace

__all__ = ["MoeLayerPlan"]


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
