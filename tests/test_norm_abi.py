"""The block norm without a GPU: bad arguments are refused before anything touches a device."""
import ctypes as C

import pytest
import torch

from moe_ffn_layer_fp32_b200 import _lib, build

P, FAR = 1 << 20, 1 << 32


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def args(**kw):
    d = dict(rows=4, d=256, r_type=1, y_type=0, gate_col=1, gate_row=0, residual_scale=1.0, eps=1e-6, r=P, ldr=256, y=FAR,
             ldy=256, w_post=2 * FAR, gate=3 * FAR, w_pre=4 * FAR, r_out=5 * FAR, ldo=256, x=6 * FAR, xq=7 * FAR, sx=8 * FAR)
    d.update(kw)
    return _lib.Norm(**d)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), b"rows"), (dict(d=0), b"d="), (dict(d=260), b"d="), (dict(d=8200), b"d="), (dict(r_type=2), b"r_type"),
    (dict(y_type=-1), b"y_type"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"), (dict(r=None), b"r is NULL"),
    (dict(y=None), b"need y"), (dict(y=None, w_post=None), b"need y"), (dict(w_pre=None), b"need w_pre"),
    (dict(x=None, xq=None, sx=None), b"needs x"), (dict(sx=None), b"together"), (dict(xq=None), b"together"),
    (dict(r_out=None, w_pre=None, x=None, xq=None, sx=None), b"no output"), (dict(ldr=248), b"r must"), (dict(ldr=260), b"r must"),
    (dict(ldy=258), b"y must"), (dict(ldo=0), b"r_out must"), (dict(y=FAR + 8), b"y must"), (dict(gate_col=2), b"gate_col"),
    (dict(gate_row=-4), b"gate_row"), (dict(gate_row=6), b"gate"), (dict(gate=3 * FAR + 4), b"gate"),
    (dict(gate=3 * FAR + 2, gate_col=0), b"gate"), (dict(w_post=2 * FAR + 4), b"aligned"), (dict(x=6 * FAR + 8), b"aligned"),
    (dict(sx=8 * FAR + 2), b"sx"), (dict(r_out=P + 16), b"overlaps an input"), (dict(r_out=P, ldo=264), b"overlaps an input"),
    (dict(x=FAR + 16), b"overlaps an input"), (dict(sx=4 * FAR + 16), b"overlaps an input"), (dict(xq=6 * FAR + 64), b"two outputs"),
    (dict(sx=7 * FAR + 1000), b"two outputs")])
def test_refuses(L, kw, word):
    assert L.mmoe_block_norm(C.byref(args(**kw)), None) == 1
    assert word in L.mmoe_last_error()


def test_null_and_nothing(L):
    assert L.mmoe_block_norm(None, None) == 1
    assert L.mmoe_block_norm(C.byref(args(rows=0, r=None)), None) == 0


def test_wrapper_refuses():
    from moe_ffn_layer_fp32_b200.norm import block_norm
    r, y, w = torch.zeros(4, 64), torch.zeros(4, 64), torch.ones(64)
    for bad in (lambda: block_norm(r, y), lambda: block_norm(r.half(), y), lambda: block_norm(r, y[:3]),
                lambda: block_norm(r, y.half()), lambda: block_norm(r, y, post_weight=w[:32]),
                lambda: block_norm(r, y, gate=torch.ones(3, 1)), lambda: block_norm(r, y, gate=torch.ones(64).double()),
                lambda: block_norm(r, y, gate=torch.ones(4, 128)[:, ::2]), lambda: block_norm(r, y, quantize=True),
                lambda: block_norm(r, y, out_residual=torch.zeros(4, 64, dtype=torch.bfloat16)),
                lambda: block_norm(torch.zeros(64, 4).t(), y)):
        with pytest.raises(ValueError):
            bad()
