"""What the operators' wrappers share: devices, streams and checks of tensors."""
from __future__ import annotations

import torch

from . import _lib

TYPE = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def same_device(x: torch.Tensor, *others) -> None:
    """x is a CUDA tensor and the others (None is skipped) are on its device."""
    at = x.get_device()
    if at < 0 or not x.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors on {x.device} and {t.device}: one device is needed")


def rows_of(t: torch.Tensor, cols: int, name: str) -> int:
    """t is [rows, cols] with unit stride along the row and rows that do not overlap; the elements between rows."""
    if t.dim() == 2:
        (rows, n), (step, unit) = t.shape, t.stride()
        if n == cols and (unit == 1 or cols == 1):
            if rows <= 1:
                return cols
            if step >= cols:
                return step
    raise ValueError(f"{name} must be [rows, {cols}] with contiguous rows")


def empty(x: torch.Tensor, rows: int, cols: int, dtype: torch.dtype) -> torch.Tensor:
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=x.device)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None


def on(x: torch.Tensor, stream):
    """(context, stream pointer) to run on x's device: inside the context (None: nothing to enter) that device is
    current and, where a stream was given, so is that stream, so that tensors allocated there belong to it."""
    if stream is None:
        at = x.get_device()
        return (None if at == _current_device() else torch.cuda.device(at)), _raw_stream(at)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def run(x: torch.Tensor, stream, call, *args):
    """call(stream pointer, *args) as `on` says."""
    context, pointer = on(x, stream)
    if context is None:
        return call(pointer, *args)
    with context:
        return call(pointer, *args)
