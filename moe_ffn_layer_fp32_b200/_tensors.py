"""What the operators' wrappers share: devices, streams and checks of tensors."""
from __future__ import annotations

import contextlib

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
    need(x.is_cuda, "tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.device != x.device:
            raise ValueError(f"tensors on {x.device} and {t.device}: one device is needed")


def rows_of(t: torch.Tensor, cols: int, name: str) -> None:
    """t is [rows, cols] with unit stride along the row and rows that do not overlap."""
    need(t.dim() == 2 and t.shape[1] == cols and (cols == 1 or t.stride(1) == 1)
         and (t.shape[0] <= 1 or t.stride(0) >= cols), f"{name} must be [rows, {cols}] with contiguous rows")


def row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


_NOTHING = contextlib.nullcontext()


def on(x: torch.Tensor, stream):
    """(context, stream pointer) to run on x's device: inside the context that device is current and, where a stream
    was given, so is that stream, so that tensors allocated there belong to it."""
    if stream is None:
        ptr = torch.cuda.current_stream(x.device).cuda_stream
        return (_NOTHING if x.device.index == torch.cuda.current_device() else torch.cuda.device(x.device)), ptr
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    need(stream.device == x.device, f"the stream is on {stream.device}, the tensors on {x.device}")
    return torch.cuda.stream(stream), stream.cuda_stream
