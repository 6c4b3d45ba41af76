"""The e4m3 MoE layer without a GPU: bad configurations and buffers are refused before anything touches a device."""
import ctypes as C

import pytest
import torch

from moe_ffn_layer_fp32_b200 import _lib, build

FAR = 1 << 32
D, HID, SH, E, K, T = 256, 128, 96, 8, 2, 5
CONFIG = dict(d=D, E=E, k=K, h=HID, hs=SH, group=128, max=64, gating=0, bias=0, flags=0)
NAMES = [n for n, _ in _lib.FP8Weights._fields_]


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def config(**kw):
    c = {**CONFIG, **kw}
    return _lib.Config(c["d"], c["E"], c["k"], c["h"], c["hs"], c["group"], c["max"], c["gating"], c["bias"], c["flags"])


def refuse(L, status, word):
    assert status == 1
    assert word in L.mmoe_last_error()


BAD_CONFIG = [
    (dict(d=32), b"d_model"), (dict(d=272), b"d_model"), (dict(d=8224), b"d_model"), (dict(E=0), b"n_experts"),
    (dict(E=65), b"n_experts"), (dict(k=0), b"top_k"), (dict(k=9), b"top_k"), (dict(E=64, k=9), b"top_k"),
    (dict(h=16), b"expert_hidden"), (dict(h=144), b"expert_hidden"), (dict(h=4128), b"expert_hidden"),
    (dict(hs=0), b"shared_hidden"), (dict(hs=100), b"shared_hidden"), (dict(group=64), b"group_size"),
    (dict(max=0), b"max_tokens"), (dict(gating=3), b"gating"), (dict(bias=2), b"has_router_bias"), (dict(flags=1), b"flags")]


@pytest.mark.parametrize("kw,word", BAD_CONFIG)
def test_config_refused(L, kw, word):
    n = C.c_size_t()
    refuse(L, L.mmoe_fp8_workspace(C.byref(config(**kw)), 1, C.byref(n)), word)
    refuse(L, forward(L, cfg=config(**kw)), word)


def test_workspace(L):
    n, c = C.c_size_t(7), config(max=20)
    assert L.mmoe_fp8_workspace(C.byref(c), 0, C.byref(n)) == 0 and n.value == 0
    last = 0
    for t in (1, 2, 8, 20):
        assert L.mmoe_fp8_workspace(C.byref(c), t, C.byref(n)) == 0 and n.value > last
        last = n.value
    refuse(L, L.mmoe_fp8_workspace(C.byref(c), 21, C.byref(n)), b"T=21")
    refuse(L, L.mmoe_fp8_workspace(C.byref(c), -1, C.byref(n)), b"T=-1")
    refuse(L, L.mmoe_fp8_workspace(C.byref(c), 1, None), b"NULL")
    refuse(L, L.mmoe_fp8_workspace(None, 1, C.byref(n)), b"NULL")
    refuse(L, L.mmoe_fp8_workspace(C.byref(config()), 65, C.byref(n)), b"T=65")


def forward(L, cfg=None, **kw):
    a = dict(x=20 * FAR, T=T, y=21 * FAR, t=1, idx=22 * FAR, gate=23 * FAR, counts=24 * FAR, ws=25 * FAR, wb=1 << 20)
    w = {n: (i + 1) * FAR for i, n in enumerate(NAMES)}
    for n, v in kw.items():
        (w if n in w else a)[n] = v
    weights = None if a.pop("no_weights", False) else C.byref(_lib.FP8Weights(*[w[n] for n in NAMES]))
    cfg = config() if cfg is None else cfg
    return L.mmoe_forward_fp8(C.byref(cfg), weights, a["x"], a["T"], a["y"], a["t"], a["idx"], a["gate"], a["counts"], a["ws"],
                              a["wb"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T=-1"), (dict(T=65), b"T=65"), (dict(t=2), b"y_type"), (dict(no_weights=True), b"weights is NULL"),
    (dict(x=None), b"NULL"), (dict(y=None), b"NULL"), (dict(x=20 * FAR + 8), b"aligned"), (dict(y=21 * FAR + 1), b"aligned"),
    (dict(idx=22 * FAR + 2), b"aligned"), (dict(gate=23 * FAR + 1), b"aligned"), (dict(counts=24 * FAR + 3), b"aligned"),
    (dict(ws=None), b"workspace"), (dict(ws=25 * FAR + 128), b"workspace"), (dict(wb=100), b"workspace"),
    (dict(y=20 * FAR), b"overlaps"), (dict(idx=21 * FAR + 64), b"overlaps"), (dict(counts=22 * FAR), b"overlaps"),
    (dict(ws=20 * FAR), b"overlaps"), (dict(y=25 * FAR + 256), b"overlaps"), (dict(w_gate_up=FAR * 3 + 8), b"aligned"),
    (dict(s_down=FAR * 6 + 2), b"aligned"), (dict(y=3 * FAR + E * 2 * HID * D - 4), b"overlaps"),
    (dict(gate=5 * FAR + E * D * HID - 4), b"overlaps")]
    + [({n: None}, b"NULL") for n in NAMES if n != "router_bias"])
def test_forward_refuses(L, kw, word):
    refuse(L, forward(L, **kw), word)


def test_router_bias_where_the_config_has_one(L):
    refuse(L, forward(L, cfg=config(bias=1), router_bias=None), b"router_bias")
    refuse(L, forward(L, cfg=config(bias=1), idx=2 * FAR + 4 * E - 4), b"overlaps")


def test_no_tokens_is_a_no_op(L):
    assert forward(L, T=0, x=None, y=None, ws=None, wb=0) == 0


def test_layer_refuses():
    from moe_ffn_layer_fp32_b200 import fp8
    with pytest.raises(_lib.MMoEError, match="d_model"):
        fp8.FP8MoELayer(100, 128)
    layer = fp8.FP8MoELayer(256, 128, n_experts=4, top_k=2)
    with pytest.raises(ValueError, match="load"):
        layer.forward(torch.zeros(1, 256, dtype=torch.bfloat16))
    e4m3 = torch.float8_e4m3fn
    z = lambda *s: torch.zeros(s)
    q = lambda *s: torch.zeros(s, dtype=torch.uint8).view(e4m3)
    good = [z(256, 4), None, q(4, 256, 256), z(4, 2, 2), q(4, 256, 128), z(4, 2, 1), q(256, 256), z(2, 2), q(256, 128), z(2, 1)]
    with pytest.raises(ValueError, match="CUDA"):
        layer.load(*good)
    for i, bad in ((0, z(4, 256)), (1, z(4)), (2, q(4, 256, 128)), (3, z(4, 1, 2)), (4, z(4, 256, 128)), (5, z(4, 1, 2)),
                   (6, q(256, 512)[:, ::2]), (7, z(2, 2).double()), (8, q(1, 256, 128)), (9, None)):
        with pytest.raises(ValueError):
            layer.load(*good[:i], bad, *good[i + 1:])
