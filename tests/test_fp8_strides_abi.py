"""Strides that no buffer has are refused before sizes are computed from them."""
import ctypes as C

import pytest

from moe_ffn_layer_fp32_b200 import _lib, build

P, FAR, BIG = 1 << 20, 1 << 32, 1 << 62


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def refuse(L, status, word):
    assert status == 1 and word in L.mmoe_last_error()


@pytest.mark.parametrize("ld", [BIG, (1 << 36) + 8])
def test_products_and_quantiser(L, ld):
    refuse(L, L.mmoe_gemm_fp8(P, 3 * FAR, 5, FAR, 2 * FAR, 100, 256, 4 * FAR, 1, ld, None), b"ldy")
    refuse(L, L.mmoe_gemm_fp8_grouped(P, 3 * FAR, 5, 5 * FAR, 2, FAR, 2 * FAR, 100, 256, 4 * FAR, 1, ld, None), b"ldy")
    refuse(L, L.mmoe_linear_fp8(P, 5, ld, FAR, 2 * FAR, 100, 256, 4 * FAR, 1, 100, None, 0, None), b"ldx")
    refuse(L, L.mmoe_quantize_fp8_rows(P, 1, 5, 256, ld, FAR, 2 * FAR, None), b"ldx")


@pytest.mark.parametrize("name,word", [("ldr", b"r must"), ("ldy", b"y must"), ("ldo", b"r_out must"), ("gate_row", b"gate_row")])
def test_norm(L, name, word):
    a = dict(rows=4, d=256, r_type=1, y_type=0, gate_col=1, gate_row=0, residual_scale=1.0, eps=1e-6, r=P, ldr=256, y=FAR,
             ldy=256, w_post=2 * FAR, gate=3 * FAR, w_pre=4 * FAR, r_out=5 * FAR, ldo=256, x=6 * FAR, xq=7 * FAR, sx=8 * FAR)
    a[name] = BIG
    refuse(L, L.mmoe_block_norm(C.byref(_lib.Norm(**a)), None), word)
