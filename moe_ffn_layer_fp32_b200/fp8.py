"""8-bit floating-point (e4m3) operators with one FP32 scale per block of 128: quantisers, matrix products and the MoE
layer on such weights.

Thin wrappers over the C ABI (include/mmoe.h): PyTorch provides device memory and streams, every step runs in
libmmoe.so.  Codes are ``torch.float8_e4m3fn`` tensors.  A tensor allocated here belongs to ``stream`` (the current
stream of the input's device by default).
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import check, lib
from ._tensors import E4M3, TYPE, blocks, empty, need, rows_of, run, same_device


def _typed(t: torch.Tensor, name: str) -> int:
    need(t.dtype in TYPE, f"{name} must be float32 or bfloat16")
    return TYPE[t.dtype]


def _scales(s: torch.Tensor, shape: tuple, name: str) -> None:
    if s.dtype != torch.float32 or s.shape != shape or not s.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 of shape {shape}")


def _codes(q: torch.Tensor, dim: int, name: str) -> None:
    if q.dtype != E4M3 or q.dim() != dim or not q.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dim}-D float8_e4m3fn tensor")


def _output(y, M: int, N: int, out_dtype, x: torch.Tensor):
    """y, its type and the elements between its rows."""
    if y is None:
        if out_dtype not in TYPE:
            raise ValueError("out_dtype must be float32 or bfloat16")
        return empty(x, M, N, out_dtype), TYPE[out_dtype], N
    if y.dtype not in TYPE or y.dim() != 2 or y.shape[0] != M:
        raise ValueError(f"y must be a float32 or bfloat16 tensor of {M} rows")
    return y, TYPE[y.dtype], rows_of(y, N, "y")


def check_timeouts(device=None) -> None:
    """Raises MMoEError (TIMEOUT), once, where a bounded wait of a product or layer call on ``device`` (default: the
    current one) has given up.  The next such call would raise it too; this is for replays of captured graphs and for
    the end of a program, and knows of work that has ended: synchronise first."""
    with torch.cuda.device(device):
        check(lib().mmoe_fp8_status())


def quantize_fp8_rows(x: torch.Tensor, *, stream=None):
    """x [rows, K] (float32 or bfloat16, rows contiguous, K a multiple of 8) -> (codes [rows, K], scales
    [rows, ceil(K / 128)])."""
    need(x.dim() == 2, "x must be 2-D")
    M, K = x.shape
    ldx, kind = rows_of(x, K, "x"), _typed(x, "x")
    same_device(x)

    def call(st):
        q, s = empty(x, M, K, E4M3), empty(x, M, blocks(K), torch.float32)
        check(lib().mmoe_quantize_fp8_rows(x.data_ptr(), kind, M, K, ldx, q.data_ptr(), s.data_ptr(), st))
        return q, s

    return run(x, stream, call)


def quantize_fp8_blocks(w: torch.Tensor, *, stream=None):
    """w [..., N, K] (float32 or bfloat16, contiguous, K a multiple of 8) -> (codes [..., N, K], scales
    [..., ceil(N / 128), ceil(K / 128)])."""
    need(w.dim() >= 2 and w.is_contiguous(), "w must be contiguous with at least two dimensions")
    kind = _typed(w, "w")
    same_device(w)
    N, K = w.shape[-2:]
    batch = w.shape[:-2].numel()

    def call(st):
        q = torch.empty(w.shape, dtype=E4M3, device=w.device)
        s = torch.empty((*w.shape[:-2], blocks(N), blocks(K)), dtype=torch.float32, device=w.device)
        check(lib().mmoe_quantize_fp8_blocks(w.data_ptr(), kind, batch, N, K, q.data_ptr(), s.data_ptr(), st))
        return q, s

    return run(w, stream, call)


def gemm_fp8(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None, *,
             out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y [M, N] = the product of quantised rows xq [M, K] and weights wq [N, K] (K a multiple of 16); y may be given
    (float32 or bfloat16, rows contiguous)."""
    _codes(xq, 2, "xq")
    _codes(wq, 2, "wq")
    (M, K), (N, Kw) = xq.shape, wq.shape
    if Kw != K:
        raise ValueError("xq and wq must have the same K")
    _scales(sx, (M, blocks(K)), "sx")
    _scales(sw, (blocks(N), blocks(K)), "sw")
    same_device(xq, sx, wq, sw, y)
    return run(xq, stream, _gemm, xq, sx, wq, sw, y, out_dtype, M, N, K)


def _gemm(st, xq, sx, wq, sw, y, out_dtype, M, N, K):
    y, kind, ldy = _output(y, M, N, out_dtype, xq)
    check(lib().mmoe_gemm_fp8(xq.data_ptr(), sx.data_ptr(), M, wq.data_ptr(), sw.data_ptr(), N, K, y.data_ptr(), kind, ldy, st))
    return y


def grouped_gemm_fp8(xq: torch.Tensor, sx: torch.Tensor, offsets: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                     y: torch.Tensor | None = None, *, out_dtype: torch.dtype = torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """Rows offsets[g] .. offsets[g + 1] - 1 of xq [M, K] times weights wq[g] of wq [G, N, K]; offsets int32 [G + 1] on
    the device.  Rows outside [offsets[0], offsets[G]) of a given y stay as they were (of a new one: undefined)."""
    _codes(xq, 2, "xq")
    _codes(wq, 3, "wq")
    (M, K), (G, N, Kw) = xq.shape, wq.shape
    if Kw != K:
        raise ValueError("xq and wq must have the same K")
    _scales(sx, (M, blocks(K)), "sx")
    _scales(sw, (G, blocks(N), blocks(K)), "sw")
    if offsets.dtype != torch.int32 or offsets.shape != (G + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets must be contiguous int32 of shape ({G + 1},)")
    same_device(xq, sx, wq, sw, offsets, y)
    return run(xq, stream, _grouped, xq, sx, offsets, wq, sw, y, out_dtype, M, G, N, K)


def _grouped(st, xq, sx, offsets, wq, sw, y, out_dtype, M, G, N, K):
    y, kind, ldy = _output(y, M, N, out_dtype, xq)
    check(lib().mmoe_gemm_fp8_grouped(xq.data_ptr(), sx.data_ptr(), M, offsets.data_ptr(), G, wq.data_ptr(), sw.data_ptr(),
                                      N, K, y.data_ptr(), kind, ldy, st))
    return y


def linear_fp8(x: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, y: torch.Tensor | None = None, *,
               out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """quantize_fp8_rows of x [M, K] (bfloat16, rows contiguous), then gemm_fp8: y [M, N].  Up to 64 rows are one
    launch."""
    _codes(wq, 2, "wq")
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    (M, K), (N, Kw) = x.shape, wq.shape
    if Kw != K:
        raise ValueError("x and wq must have the same K")
    ldx = rows_of(x, K, "x")
    _scales(sw, (blocks(N), blocks(K)), "sw")
    same_device(x, wq, sw, y)
    return run(x, stream, _linear, x, ldx, wq, sw, y, out_dtype, M, N, K)


def _linear(st, x, ldx, wq, sw, y, out_dtype, M, N, K):
    y, kind, ldy = _output(y, M, N, out_dtype, x)
    size, room, at = 0, None, None
    if M > 64:
        size = 16 * -(-M * blocks(K) // 4) + M * K  # mmoe_linear_fp8_workspace
        room = empty(x, 1, size, torch.uint8)
        at = room.data_ptr()
    check(lib().mmoe_linear_fp8(x.data_ptr(), M, ldx, wq.data_ptr(), sw.data_ptr(), N, K, y.data_ptr(), kind, ldy, at, size,
                                st))
    return y


def _optional(t: torch.Tensor | None, shape: tuple, dtype, name: str):
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of shape {shape}")
    return t.data_ptr()


class FP8MoELayer:
    """The MoE feed-forward layer (Eq. (*) of the MobileMoE pages) on e4m3 weights, for up to 64 tokens a call (more are
    refused: a prompt takes calls of 64, each of which reads the selected experts' weights again).

    ``load`` keeps the caller's tensors and reads them in place; every ``forward`` allocates its own workspace, so that
    calls on several streams, and captured graphs, do not share one."""

    def __init__(self, d_model: int, expert_hidden: int, *, shared_hidden: int | None = None, n_experts: int = 60,
                 top_k: int = 4, max_tokens: int = 64, gating: int = 0, has_router_bias: bool = False):
        self.cfg = _lib.Config(d_model, n_experts, top_k, expert_hidden,
                               expert_hidden if shared_hidden is None else shared_hidden, 128, max_tokens, gating,
                               int(has_router_bias), 0)
        self._sizes = d_model, top_k, n_experts
        self._config = C.byref(self.cfg)
        self._keep = None
        self._room: dict[int, int] = {}  # workspace bytes for a number of tokens
        self._workspace_bytes(0)         # checks the config

    @property
    def d_model(self) -> int:
        return self.cfg.d_model

    def _workspace_bytes(self, T: int) -> int:
        if T not in self._room:
            n = C.c_size_t()
            check(lib().mmoe_fp8_workspace(C.byref(self.cfg), T, C.byref(n)))
            self._room[T] = n.value
        return self._room[T]

    def load(self, w_router, router_bias, w_gate_up, s_gate_up, w_down, s_down, w_shared_gate_up, s_shared_gate_up,
             w_shared_down, s_shared_down) -> None:
        """Weights in the layout of include/mmoe.h (mmoe_fp8_weights), contiguous CUDA tensors on one device."""
        c = self.cfg
        d, h, hs, E = c.d_model, c.expert_hidden, c.shared_hidden, c.n_experts
        need((router_bias is not None) == bool(c.has_router_bias), "router_bias must be given exactly where the layer has one")
        for t, shape, dtype, name in (
                (w_router, (d, E), torch.float32, "w_router"), (router_bias, (E,), torch.float32, "router_bias"),
                (w_gate_up, (E, 2 * h, d), E4M3, "w_gate_up"), (w_down, (E, d, h), E4M3, "w_down"),
                (s_gate_up, (E, 2 * blocks(h), blocks(d)), torch.float32, "s_gate_up"),
                (s_down, (E, blocks(d), blocks(h)), torch.float32, "s_down"),
                (w_shared_gate_up, (2 * hs, d), E4M3, "w_shared_gate_up"), (w_shared_down, (d, hs), E4M3, "w_shared_down"),
                (s_shared_gate_up, (2 * blocks(hs), blocks(d)), torch.float32, "s_shared_gate_up"),
                (s_shared_down, (blocks(d), blocks(hs)), torch.float32, "s_shared_down")):
            need(t is not None or name == "router_bias", f"{name} must be given")
            _optional(t, shape, dtype, name)
        keep = (w_router, router_bias, w_gate_up, s_gate_up, w_down, s_down, w_shared_gate_up, s_shared_gate_up,
                w_shared_down, s_shared_down)
        same_device(*keep)
        self._keep = keep
        self._weights = _lib.FP8Weights(*[None if t is None else t.data_ptr() for t in keep])
        self._pointers = C.byref(self._weights)

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, *, out_dtype: torch.dtype = torch.float32, stream=None,
                topk_idx=None, topk_gate=None, expert_counts=None) -> torch.Tensor:
        """y [T, d] (given, or new of out_dtype: float32 or bfloat16) from x [T, d] (bfloat16, contiguous)."""
        if self._keep is None:
            raise ValueError("the layer has no weights: call load() first")
        d, k, E = self._sizes
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != d or not x.is_contiguous():
            raise ValueError("x must be a contiguous [T, d_model] bfloat16 tensor")
        T = x.shape[0]
        idx, gate = _optional(topk_idx, (T, k), torch.int32, "topk_idx"), _optional(topk_gate, (T, k), torch.float32, "topk_gate")
        counts = _optional(expert_counts, (E + 1,), torch.int32, "expert_counts")
        same_device(x, self._keep[0], y, topk_idx, topk_gate, expert_counts)
        return run(x, stream, self._forward, x, T, y, out_dtype, idx, gate, counts)

    def _forward(self, st, x, T, y, out_dtype, idx, gate, counts):
        d = self._sizes[0]
        if y is None:
            if out_dtype not in TYPE:
                raise ValueError("out_dtype must be float32 or bfloat16")
            y = empty(x, T, d, out_dtype)
        elif y.dtype not in TYPE or y.shape != (T, d) or not y.is_contiguous():
            raise ValueError("y must be a contiguous [T, d_model] float32 or bfloat16 tensor")
        size = self._room.get(T)
        if size is None:
            size = self._workspace_bytes(T)
        room = empty(x, 1, size, torch.uint8)
        check(lib().mmoe_forward_fp8(self._config, self._pointers, x.data_ptr(), T, y.data_ptr(), TYPE[y.dtype], idx, gate,
                                     counts, room.data_ptr(), size, st))
        return y

    __call__ = forward
