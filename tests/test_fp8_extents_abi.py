"""Buffers that a call of the e4m3 operators would write over, refused before anything touches a device."""
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
