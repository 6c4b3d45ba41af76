"""The e4m3 operators without a GPU: bad arguments are refused before anything touches a device."""
import ctypes as C

import pytest
import torch

from moe_ffn_layer_fp32_b200 import _lib, build

P = 1 << 20  # a well aligned address that nothing dereferences
FAR = 1 << 32


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def refuse(L, status, word):
    assert status == 1
    assert word in L.mmoe_last_error()


def rows(L, x=P, t=1, M=4, K=256, ldx=256, q=FAR, s=2 * FAR):
    return L.mmoe_quantize_fp8_rows(x, t, M, K, ldx, q, s, None)


@pytest.mark.parametrize("kw,word", [
    (dict(M=-1), b"rows"), (dict(K=0), b"K="), (dict(K=12), b"K="), (dict(K=1 << 21), b"K="), (dict(t=2), b"x_type"),
    (dict(ldx=248), b"ldx"), (dict(ldx=260), b"ldx"), (dict(x=None), b"NULL"), (dict(q=None), b"NULL"),
    (dict(s=None), b"NULL"), (dict(x=P + 2), b"aligned"), (dict(q=FAR + 4), b"aligned"), (dict(s=FAR * 2 + 2), b"aligned"),
    (dict(q=P + 256), b"overlap"), (dict(s=FAR + 64), b"overlap")])
def test_quantize_rows_refuses(L, kw, word):
    refuse(L, rows(L, **kw), word)


def test_quantize_nothing_is_a_no_op(L):
    assert rows(L, M=0, x=None, q=None, s=None) == 0
    assert L.mmoe_quantize_fp8_blocks(None, 0, 0, 128, 128, None, None, None) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(batch=-1), b"batch"), (dict(N=0), b"N="), (dict(K=20), b"K="), (dict(t=-1), b"w_type"), (dict(w=None), b"NULL"),
    (dict(w=P + 8), b"aligned"), (dict(q=P), b"overlap"), (dict(batch=1 << 30, N=1 << 20), b"blocks")])
def test_quantize_blocks_refuses(L, kw, word):
    a = dict(w=P, t=0, batch=2, N=200, K=256, q=FAR, s=2 * FAR)
    a.update(kw)
    refuse(L, L.mmoe_quantize_fp8_blocks(a["w"], a["t"], a["batch"], a["N"], a["K"], a["q"], a["s"], None), word)


PRODUCT = [
    (dict(M=-1), b"M="), (dict(M=1 << 31), b"M="), (dict(N=0), b"N="), (dict(K=24), b"K="), (dict(K=0), b"K="),
    (dict(t=7), b"y_type"), (dict(ldy=99), b"ldy"), (dict(w=None), b"NULL"), (dict(sw=None), b"NULL"),
    (dict(y=None), b"NULL"), (dict(w=FAR + 8), b"aligned"), (dict(y=4 * FAR + 1), b"aligned"), (dict(y=FAR), b"overlaps"),
    (dict(y=2 * FAR), b"overlaps")]
CODES = [(dict(a=None), b"NULL"), (dict(sa=None), b"NULL"), (dict(a=P + 8), b"aligned"), (dict(y=P), b"overlaps"),
         (dict(y=3 * FAR), b"overlaps")]
DEFAULT = dict(a=P, sa=3 * FAR, M=5, w=FAR, sw=2 * FAR, N=100, K=256, y=4 * FAR, t=1, ldy=100)


@pytest.mark.parametrize("kw,word", PRODUCT + CODES)
def test_gemm_refuses(L, kw, word):
    d = {**DEFAULT, **kw}
    refuse(L, L.mmoe_gemm_fp8(d["a"], d["sa"], d["M"], d["w"], d["sw"], d["N"], d["K"], d["y"], d["t"], d["ldy"], None), word)


@pytest.mark.parametrize("kw,word", PRODUCT + CODES + [
    (dict(G=0), b"groups"), (dict(G=1025), b"groups"), (dict(off=None), b"offsets"), (dict(off=5 * FAR + 2), b"offsets"),
    (dict(off=4 * FAR + 40), b"offsets"), (dict(G=1024, N=1 << 20, K=1 << 20, ldy=1 << 20), b"too many")])
def test_grouped_gemm_refuses(L, kw, word):
    d = {**DEFAULT, "G": 3, "off": 5 * FAR, **kw}
    refuse(L, L.mmoe_gemm_fp8_grouped(d["a"], d["sa"], d["M"], d["off"], d["G"], d["w"], d["sw"], d["N"], d["K"], d["y"],
                                      d["t"], d["ldy"], None), word)


@pytest.mark.parametrize("kw,word", PRODUCT + [
    (dict(x=None), b"x is NULL"), (dict(x=P + 2), b"aligned"), (dict(ldx=248), b"ldx"), (dict(ldx=260), b"ldx"),
    (dict(y=P), b"overlap"), (dict(M=65, ws=None), b"workspace"), (dict(M=65, ws=6 * FAR + 4), b"workspace"),
    (dict(M=65, wb=65 * 256 + 65 * 8 - 1), b"workspace"), (dict(M=65, ws=4 * FAR), b"workspace")])
def test_linear_refuses(L, kw, word):
    d = {**DEFAULT, "x": P, "ldx": 256, "ws": 6 * FAR, "wb": 1 << 20, **kw}
    refuse(L, L.mmoe_linear_fp8(d["x"], d["M"], d["ldx"], d["w"], d["sw"], d["N"], d["K"], d["y"], d["t"], d["ldy"], d["ws"],
                                d["wb"], None), word)


def test_no_rows_is_a_no_op(L):
    assert L.mmoe_gemm_fp8(None, None, 0, None, None, 8, 16, None, 0, 8, None) == 0
    assert L.mmoe_gemm_fp8_grouped(None, None, 0, None, 1, None, None, 8, 16, None, 0, 8, None) == 0
    assert L.mmoe_linear_fp8(None, 0, 16, None, None, 8, 16, None, 0, 8, None, 0, None) == 0


def test_linear_workspace(L):
    n = C.c_size_t(7)
    assert L.mmoe_linear_fp8_workspace(64, 1024, C.byref(n)) == 0 and n.value == 0
    assert L.mmoe_linear_fp8_workspace(65, 144, C.byref(n)) == 0 and n.value == 65 * 144 + 528
    refuse(L, L.mmoe_linear_fp8_workspace(65, 144, None), b"NULL")
    refuse(L, L.mmoe_linear_fp8_workspace(65, 8, C.byref(n)), b"K=")


def test_wrappers_refuse():
    from moe_ffn_layer_fp32_b200 import fp8
    e4m3 = torch.float8_e4m3fn
    q, s = torch.zeros(4, 256, dtype=torch.uint8).view(e4m3), torch.zeros(4, 2)
    w, sw = torch.zeros(100, 256, dtype=torch.uint8).view(e4m3), torch.zeros(1, 2)
    for bad in (lambda: fp8.gemm_fp8(q, s, w, sw),                          # not on a GPU
                lambda: fp8.gemm_fp8(q.view(torch.uint8), s, w, sw),        # not codes
                lambda: fp8.gemm_fp8(q, s, w[:, :240], sw),                 # strided weights
                lambda: fp8.gemm_fp8(q, s[:, :1], w, sw),                   # too few scales
                lambda: fp8.gemm_fp8(q, s, w, sw.double()),                 # scales of another type
                lambda: fp8.gemm_fp8(q, s, w, sw, torch.zeros(4, 99)),      # output of another width
                lambda: fp8.grouped_gemm_fp8(q, s, torch.zeros(3, dtype=torch.int64), w[None], sw[None]),
                lambda: fp8.linear_fp8(torch.zeros(4, 256), w, sw),         # x is not bfloat16
                lambda: fp8.linear_fp8(torch.zeros(256, 4, dtype=torch.bfloat16).t(), w, sw),  # rows not contiguous
                lambda: fp8.quantize_fp8_rows(torch.zeros(4, 256, dtype=torch.float16)),
                lambda: fp8.quantize_fp8_rows(torch.zeros(4, 256)),
                lambda: fp8.quantize_fp8_blocks(torch.zeros(256))):
        with pytest.raises(ValueError):
            bad()
