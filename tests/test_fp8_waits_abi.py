"""The wait limits of the e4m3 operators without a GPU: arguments, and what a status query says before any call."""
import pytest
import torch

from moe_ffn_layer_fp32_b200 import _lib, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


@pytest.mark.parametrize("clocks,stall,word", [(-1, 0, b"clocks"), (0, -1, b"stall_next"), (0, 3, b"stall_next")])
def test_refuses(L, clocks, stall, word):
    assert L.mmoe_debug_fp8_waits(clocks, stall) == 1
    assert word in L.mmoe_last_error()


def test_accepts_and_restores(L):
    assert L.mmoe_debug_fp8_waits(40_000, 2) == 0
    assert L.mmoe_debug_fp8_waits(0, 0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_status_without_a_device_is_a_cuda_error(L):
    assert L.mmoe_fp8_status() == 4
