"""Zeros keep their sign in e4m3 codes: the code of v is that of v / s, bit for bit, -0 and what rounds to it included."""
import pytest
import torch

from tests import fp8_util as U
from tests.test_gpu_fp8 import fp8, gen  # noqa: F401 (a fixture)
from tests.test_gpu_norm import norm  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def code_bytes(q):
    return q.to(F32).to(torch.float8_e4m3fn).view(torch.uint8)


def with_zeros(m, k, seed):
    """Both zeros, and values that round to either, in blocks of every scale: divided and corrected ones."""
    x = torch.randn(m, k, generator=gen(seed)) * torch.exp2(torch.linspace(-110, 118, m).round())[:, None]
    x[:, 0::7], x[:, 3::7] = -0.0, 0.0
    x[:, 5::7] *= 2.0 ** -14
    return x


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows(fp8, dtype):  # noqa: F811
    x = with_zeros(40, 264, 1).to(dtype)
    q, s = fp8.quantize_fp8_rows(x.cuda())
    rq, rs = U.quantize_rows(x.float())
    assert torch.equal(s.cpu(), rs)
    want = code_bytes(rq)
    assert bool((want == 0x80).any()) and bool((want == 0).any())
    assert torch.equal(q.view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("power", [-100, -60, 0, 90])
def test_blocks(fp8, dtype, power):  # noqa: F811
    w = torch.randn(200, 272, generator=gen(2)) * 2.0 ** power
    w[::3, ::5], w[1::3, ::5] = -0.0, 0.0
    w[2::3, ::5] *= 2.0 ** -14
    w = w.to(dtype)
    q, s = fp8.quantize_fp8_blocks(w.cuda())
    rq, rs = U.quantize_blocks(w.float())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.view(torch.uint8).cpu(), code_bytes(rq))


@pytest.mark.parametrize("d", [136, 2048, 4104])
def test_norm_codes(norm, d):  # noqa: F811
    r = torch.randn(5, d, generator=gen(3))
    r[:, ::3], r[:, 1::3] = -0.0, 0.0
    _, x, xq, _ = norm(r.cuda(), pre_weight=torch.ones(d).cuda(), quantize=True)
    zero = (r == 0).cuda()
    assert torch.equal(torch.signbit(x)[zero], torch.signbit(r.cuda())[zero])
    assert torch.equal(xq.view(torch.uint8)[zero], torch.signbit(r.cuda())[zero].to(torch.uint8) * 0x80)


def test_codes_of_one_value_do_not_depend_on_the_scale(fp8):  # noqa: F811
    """Scales inside and outside of the range of the corrected quotient give the same codes."""
    x = torch.randn(1, 128, generator=gen(4))
    x[0, ::4], x[0, 1::4] = -0.0, 0.0
    rows = torch.cat([x * 2.0 ** e for e in (-100, -70, 0, 60, 100, 115)])
    q, _ = fp8.quantize_fp8_rows(rows.cuda())
    assert bool((q.view(torch.uint8) == q.view(torch.uint8)[2]).all())
