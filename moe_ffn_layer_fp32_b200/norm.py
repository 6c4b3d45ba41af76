"""The norms after and before a block, fused with the block's gate and the residual update (include/mmoe.h)."""
from __future__ import annotations

import ctypes as C
import struct

import torch

from . import _lib
from ._lib import check, lib
from ._tensors import E4M3, TYPE, blocks, empty, need, rows_of, run, same_device


# mmoe_norm as bytes: a third of the time that its ctypes structure takes
_FORMAT = struct.Struct("@qiiiiqffPqPqPPPPqPPP")
_ARGUMENTS = _FORMAT.pack
assert _FORMAT.size == C.sizeof(_lib.Norm)


def _weight(w: torch.Tensor | None, d: int, name: str):
    if w is None:
        return None
    if w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 of shape ({d},)")
    return w.data_ptr()


def _gate(gate: torch.Tensor | None, T: int, d: int):
    """(pointer, elements between rows, between columns) of a gate [d], [T, 1], [1, d] or [T, d]."""
    if gate is None:
        return None, 0, 0
    need(gate.dtype == torch.float32, "gate must be float32")
    shape, step = tuple(gate.shape), gate.stride()
    if len(shape) == 1:
        shape, step = (1, *shape), (0, *step)
    if len(shape) != 2 or shape[0] not in (1, T) or shape[1] not in (1, d):
        raise ValueError(f"gate must be [{d}], [{T}, 1], [1, {d}] or [{T}, {d}]")
    row = step[0] if shape[0] > 1 else 0
    col = step[1] if shape[1] > 1 else 0
    need(col in (0, 1), "gate must have contiguous rows")
    return gate.data_ptr(), row, col


def block_norm(residual: torch.Tensor, y: torch.Tensor | None = None, *, post_weight: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, residual_scale: float = 1.0, pre_weight: torch.Tensor | None = None,
               eps: float = 1e-6, out_residual: torch.Tensor | None = None, quantize: bool = False, stream=None):
    """(r', x, xq, sx) of the residual stream [T, d] (float32 or bfloat16) and a block's output y [T, d] (either type):

        z  = y * rsqrt(mean(y ** 2) + eps) * post_weight      (z = y without post_weight)
        r' = residual_scale * residual + gate * z             (gate float32: [d], [T, 1] or [T, d])
        x  = r' * rsqrt(mean(r' ** 2) + eps) * pre_weight     (bfloat16; None without pre_weight)

    xq, sx are x's e4m3 codes and scales per 128 features (None without quantize).  Without y, r' is the scaled
    residual, and None unless out_residual is given.  r' goes into out_residual (which may be ``residual`` itself) or a
    new tensor.  Nothing is rounded before the outputs."""
    if residual.dim() != 2 or residual.dtype not in TYPE:
        raise ValueError("residual must be a 2-D float32 or bfloat16 tensor")
    T, d = residual.shape
    ldr = rows_of(residual, d, "residual")
    kind, y_kind, y_at, ldy = TYPE[residual.dtype], _lib.F32, None, 0
    if y is not None:
        if y.dtype not in TYPE or y.dim() != 2 or y.shape[0] != T:
            raise ValueError(f"y must be a float32 or bfloat16 tensor of {T} rows")
        y_kind, y_at, ldy = TYPE[y.dtype], y.data_ptr(), rows_of(y, d, "y")
    out_at, ldo = None, 0
    if out_residual is not None:
        if out_residual.dtype != residual.dtype or out_residual.dim() != 2 or out_residual.shape[0] != T:
            raise ValueError("out_residual must have residual's type and rows")
        out_at, ldo = out_residual.data_ptr(), rows_of(out_residual, d, "out_residual")
    need(not quantize or pre_weight is not None, "quantize needs pre_weight")
    post, pre = _weight(post_weight, d, "post_weight"), _weight(pre_weight, d, "pre_weight")
    gate_at, gate_row, gate_col = _gate(gate, T, d)
    same_device(residual, y, post_weight, gate, pre_weight, out_residual)

    return run(residual, stream, _block_norm, residual, y, out_residual, quantize, T, d, kind, y_kind, gate_col, gate_row,
               residual_scale, eps, ldr, y_at, ldy, post, gate_at, pre, out_at, ldo)


def _block_norm(st, residual, y, out, quantize, T, d, kind, y_kind, gate_col, gate_row, scale, eps, ldr, y_at, ldy, post,
                gate_at, pre, out_at, ldo):
    if out is None and y is not None:
        out = empty(residual, T, d, residual.dtype)
        out_at, ldo = out.data_ptr(), d
    x = xq = sx = None
    x_at = xq_at = sx_at = 0
    if pre is not None:
        x = empty(residual, T, d, torch.bfloat16)
        x_at = x.data_ptr()
        if quantize:
            xq, sx = empty(residual, T, d, E4M3), empty(residual, T, blocks(d), torch.float32)
            xq_at, sx_at = xq.data_ptr(), sx.data_ptr()
    check(lib().mmoe_block_norm(_ARGUMENTS(T, d, kind, y_kind, gate_col, gate_row, scale, eps, residual.data_ptr(), ldr,
                                           y_at or 0, ldy, post or 0, gate_at or 0, pre or 0, out_at or 0, ldo, x_at, xq_at,
                                           sx_at), st))
    return out, x, xq, sx
