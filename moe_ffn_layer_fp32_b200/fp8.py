"""8-bit floating-point (e4m3) operators with one FP32 scale per block of 128: quantisers and matrix products.

Thin wrappers over the C ABI (include/mmoe.h): PyTorch provides device memory and streams, every step runs in
libmmoe.so.  Codes are ``torch.float8_e4m3fn`` tensors.  A tensor allocated here belongs to ``stream`` (the current
stream of the input's device by default).
"""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import check, lib
from ._tensors import E4M3, TYPE, blocks, need, on, row_stride, rows_of, same_device


def _typed(t: torch.Tensor, name: str) -> int:
    need(t.dtype in TYPE, f"{name} must be float32 or bfloat16")
    return TYPE[t.dtype]


def _scales(s: torch.Tensor, shape, name: str) -> None:
    need(s.dtype == torch.float32 and tuple(s.shape) == tuple(shape) and s.is_contiguous(),
         f"{name} must be contiguous float32 of shape {tuple(shape)}")


def _codes(q: torch.Tensor, dim: int, name: str) -> None:
    need(q.dtype == E4M3 and q.dim() == dim and q.is_contiguous(), f"{name} must be a contiguous {dim}-D float8_e4m3fn tensor")


def _output(y, M: int, N: int, out_dtype, x: torch.Tensor):
    if y is None:
        need(out_dtype in TYPE, "out_dtype must be float32 or bfloat16")
        return torch.empty((M, N), dtype=out_dtype, device=x.device)
    need(y.dtype in TYPE and y.shape[0] == M, f"y must be a float32 or bfloat16 tensor of {M} rows")
    rows_of(y, N, "y")
    return y


def quantize_fp8_rows(x: torch.Tensor, *, stream=None):
    """x [rows, K] (float32 or bfloat16, rows contiguous, K a multiple of 8) -> (codes [rows, K], scales
    [rows, ceil(K / 128)])."""
    need(x.dim() == 2, "x must be 2-D")
    M, K = x.shape
    rows_of(x, K, "x")
    kind = _typed(x, "x")
    same_device(x)
    ctx, st = on(x, stream)
    with ctx:
        q = torch.empty((M, K), dtype=E4M3, device=x.device)
        s = torch.empty((M, blocks(K)), dtype=torch.float32, device=x.device)
        check(lib().mmoe_quantize_fp8_rows(x.data_ptr(), kind, M, K, row_stride(x), q.data_ptr(), s.data_ptr(), st))
    return q, s


def quantize_fp8_blocks(w: torch.Tensor, *, stream=None):
    """w [..., N, K] (float32 or bfloat16, contiguous, K a multiple of 8) -> (codes [..., N, K], scales
    [..., ceil(N / 128), ceil(K / 128)])."""
    need(w.dim() >= 2 and w.is_contiguous(), "w must be contiguous with at least two dimensions")
    kind = _typed(w, "w")
    same_device(w)
    N, K = w.shape[-2:]
    batch = w.shape[:-2].numel()
    ctx, st = on(w, stream)
    with ctx:
        q = torch.empty(w.shape, dtype=E4M3, device=w.device)
        s = torch.empty((*w.shape[:-2], blocks(N), blocks(K)), dtype=torch.float32, device=w.device)
        check(lib().mmoe_quantize_fp8_blocks(w.data_ptr(), kind, batch, N, K, q.data_ptr(), s.data_ptr(), st))
    return q, s


def gemm_fp8(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None, *,
             out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y [M, N] = the product of quantised rows xq [M, K] and weights wq [N, K] (K a multiple of 16); y may be given
    (float32 or bfloat16, rows contiguous)."""
    _codes(xq, 2, "xq")
    _codes(wq, 2, "wq")
    (M, K), N = xq.shape, wq.shape[0]
    need(wq.shape[1] == K, "xq and wq must have the same K")
    _scales(sx, (M, blocks(K)), "sx")
    _scales(sw, (blocks(N), blocks(K)), "sw")
    same_device(xq, sx, wq, sw, y)
    ctx, st = on(xq, stream)
    with ctx:
        y = _output(y, M, N, out_dtype, xq)
        check(lib().mmoe_gemm_fp8(xq.data_ptr(), sx.data_ptr(), M, wq.data_ptr(), sw.data_ptr(), N, K, y.data_ptr(),
                                  TYPE[y.dtype], row_stride(y), st))
    return y


def grouped_gemm_fp8(xq: torch.Tensor, sx: torch.Tensor, offsets: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                     y: torch.Tensor | None = None, *, out_dtype: torch.dtype = torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """Rows offsets[g] .. offsets[g + 1] - 1 of xq [M, K] times weights wq[g] of wq [G, N, K]; offsets int32 [G + 1] on
    the device.  Rows outside [offsets[0], offsets[G]) of a given y stay as they were (of a new one: undefined)."""
    _codes(xq, 2, "xq")
    _codes(wq, 3, "wq")
    (M, K), (G, N) = xq.shape, wq.shape[:2]
    need(wq.shape[2] == K, "xq and wq must have the same K")
    _scales(sx, (M, blocks(K)), "sx")
    _scales(sw, (G, blocks(N), blocks(K)), "sw")
    need(offsets.dtype == torch.int32 and offsets.shape == (G + 1,) and offsets.is_contiguous(),
         f"offsets must be contiguous int32 of shape ({G + 1},)")
    same_device(xq, sx, wq, sw, offsets, y)
    ctx, st = on(xq, stream)
    with ctx:
        y = _output(y, M, N, out_dtype, xq)
        check(lib().mmoe_gemm_fp8_grouped(xq.data_ptr(), sx.data_ptr(), M, offsets.data_ptr(), G, wq.data_ptr(),
                                          sw.data_ptr(), N, K, y.data_ptr(), TYPE[y.dtype], row_stride(y), st))
    return y


def linear_fp8(x: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None, *,
               out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """quantize_fp8_rows of x [M, K] (bfloat16, rows contiguous), then gemm_fp8: y [M, N].  Up to 64 rows are one
    launch."""
    _codes(wq, 2, "wq")
    need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be a 2-D bfloat16 tensor")
    (M, K), N = x.shape, wq.shape[0]
    need(wq.shape[1] == K, "x and wq must have the same K")
    rows_of(x, K, "x")
    _scales(sw, (blocks(N), blocks(K)), "sw")
    same_device(x, wq, sw, y)
    ctx, st = on(x, stream)
    with ctx:
        y = _output(y, M, N, out_dtype, x)
        size, room, at = 0, None, None
        if M > 64:
            bytes_ = C.c_size_t()
            check(lib().mmoe_linear_fp8_workspace(M, K, C.byref(bytes_)))
            size = bytes_.value
            room = torch.empty(size, dtype=torch.uint8, device=x.device)
            at = room.data_ptr()
        check(lib().mmoe_linear_fp8(x.data_ptr(), M, row_stride(x), wq.data_ptr(), sw.data_ptr(), N, K, y.data_ptr(),
                                    TYPE[y.dtype], row_stride(y), at, size, st))
    return y
