"""The norms after and before a block, fused with the block's gate and the residual update (include/mmoe.h)."""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import check, lib
from ._tensors import E4M3, TYPE, blocks, need, on, row_stride, rows_of, same_device


def _weight(w: torch.Tensor | None, d: int, name: str):
    if w is None:
        return None
    need(w.dtype == torch.float32 and w.shape == (d,) and w.is_contiguous(), f"{name} must be contiguous float32 of shape ({d},)")
    return w.data_ptr()


def _gate(gate: torch.Tensor | None, T: int, d: int):
    """(pointer, elements between rows, between columns) of a gate [d], [T, 1], [1, d] or [T, d]."""
    if gate is None:
        return None, 0, 0
    need(gate.dtype == torch.float32, "gate must be float32")
    if gate.dim() == 1:
        gate = gate.unsqueeze(0)
    need(gate.dim() == 2 and gate.shape[0] in (1, T) and gate.shape[1] in (1, d), f"gate must be [{d}], [{T}, 1], [1, {d}] or [{T}, {d}]")
    row = gate.stride(0) if gate.shape[0] > 1 else 0
    col = gate.stride(1) if gate.shape[1] > 1 else 0
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
    need(residual.dim() == 2 and residual.dtype in TYPE, "residual must be a 2-D float32 or bfloat16 tensor")
    T, d = residual.shape
    rows_of(residual, d, "residual")
    if y is not None:
        need(y.dtype in TYPE and y.dim() == 2 and y.shape[0] == T, f"y must be a float32 or bfloat16 tensor of {T} rows")
        rows_of(y, d, "y")
    if out_residual is not None:
        need(out_residual.dtype == residual.dtype and out_residual.dim() == 2 and out_residual.shape[0] == T,
             "out_residual must have residual's type and rows")
        rows_of(out_residual, d, "out_residual")
    need(not quantize or pre_weight is not None, "quantize needs pre_weight")
    post, pre = _weight(post_weight, d, "post_weight"), _weight(pre_weight, d, "pre_weight")
    gp, gr, gc = _gate(gate, T, d)
    same_device(residual, y, post_weight, gate, pre_weight, out_residual)
    ctx, st = on(residual, stream)
    dev = residual.device
    with ctx:
        if out_residual is None and y is not None:
            out_residual = torch.empty((T, d), dtype=residual.dtype, device=dev)
        x = xq = sx = None
        if pre is not None:
            x = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
            if quantize:
                xq = torch.empty((T, d), dtype=E4M3, device=dev)
                sx = torch.empty((T, blocks(d)), dtype=torch.float32, device=dev)
        n = _lib.Norm(T, d, TYPE[residual.dtype], _lib.F32 if y is None else TYPE[y.dtype], gc, gr, residual_scale, eps,
                      residual.data_ptr(), row_stride(residual), None if y is None else y.data_ptr(),
                      0 if y is None else row_stride(y), post, gp, pre,
                      None if out_residual is None else out_residual.data_ptr(),
                      0 if out_residual is None else row_stride(out_residual), None if x is None else x.data_ptr(),
                      None if xq is None else xq.data_ptr(), None if sx is None else sx.data_ptr())
        check(lib().mmoe_block_norm(C.byref(n), st))
    return out_residual, x, xq, sx
