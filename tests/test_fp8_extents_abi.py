"""Buffers that a call of the e4m3 operators or the block norm would write over, and extents past 64 bits, are refused
before anything touches a device."""
import ctypes as C

import pytest

from moe_ffn_layer_fp32_b200 import _lib, build

P, FAR = 1 << 20, 1 << 32


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def refuse(L, status, word):
    assert status == 1
    assert word in L.mmoe_last_error()


# M = 65, K = 256: 65 x 2 scales (520 bytes, 528 with the padding), then 65 x 256 codes
@pytest.mark.parametrize("workspace", [2 * FAR, 2 * FAR - 16, 2 * FAR - 528, 2 * FAR - 528 - 65 * 256 + 16])
def test_linear_workspace_over_the_weight_scales(L, workspace):
    refuse(L, L.mmoe_linear_fp8(P, 65, 256, FAR, 2 * FAR, 100, 256, 4 * FAR, 1, 100, workspace, 1 << 20, None), b"workspace overlaps")


# (M - 1) * ld is a multiple of 2^64, so that a size computed from it in 64 bits wraps to that of one row
ROWS, LD = (1 << 28) + 1, 1 << 36


def test_product_rows_past_64_bits(L):
    y = P - 4096  # the wrapped extent would end in front of the codes at P
    refuse(L, L.mmoe_gemm_fp8(P, 3 * FAR, ROWS, FAR, 2 * FAR, 100, 256, y, 1, LD, None), b"ldy")
    refuse(L, L.mmoe_gemm_fp8_grouped(P, 3 * FAR, ROWS, 5 * FAR, 2, FAR, 2 * FAR, 100, 256, y, 1, LD, None), b"ldy")
    refuse(L, L.mmoe_linear_fp8(P, ROWS, 256, FAR, 2 * FAR, 100, 256, y, 1, LD, None, 0, None), b"ldy")
    refuse(L, L.mmoe_linear_fp8(P, ROWS, LD, FAR, 2 * FAR, 100, 256, 4 * FAR, 1, 100, None, 0, None), b"ldx")


def test_quantiser_rows_past_64_bits(L):
    refuse(L, L.mmoe_quantize_fp8_rows(P, 1, ROWS, 256, LD, FAR, 1 << 50, None), b"ldx")


@pytest.mark.parametrize("name,word", [("ldr", b" r="), ("ldy", b" y="), ("ldo", b" r_out="), ("gate_row", b"gate_row")])
def test_norm_rows_past_64_bits(L, name, word):
    a = dict(rows=ROWS, d=256, r_type=1, y_type=0, gate_col=1, gate_row=0, residual_scale=1.0, eps=1e-6, r=1 << 40, ldr=256,
             y=1 << 41, ldy=256, w_post=2 * FAR, gate=3 * FAR, w_pre=4 * FAR, r_out=1 << 42, ldo=256, x=1 << 43, xq=1 << 44,
             sx=1 << 45)
    a[name] = LD
    refuse(L, L.mmoe_block_norm(C.byref(_lib.Norm(**a)), None), word)


def test_spans_up_to_the_limit_pass(L):
    """The limit is on the product: few rows far apart, or many rows near each other, are only refused for what else is
    wrong with them."""
    refuse(L, L.mmoe_quantize_fp8_rows(P, 1, (1 << 12) + 1, 256, LD, P + 256, 1 << 60, None), b"overlap")
    refuse(L, L.mmoe_quantize_fp8_rows(P, 1, (1 << 12) + 2, 256, LD, P + 256, 1 << 60, None), b"ldx")
    refuse(L, L.mmoe_quantize_fp8_rows(P, 1, (1 << 31) - 256, 256, 256, P + 256, 1 << 60, None), b"overlap")
