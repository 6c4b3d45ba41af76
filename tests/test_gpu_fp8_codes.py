"""e4m3 codes and scales at the ends of FP32's range and on rounding borders, and grouped products in wide tiles."""
import pytest
import torch

from tests import fp8_util as U
from tests.test_gpu_fp8 import activations, codes, fp8, gen, grouped_reference, weights  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def same(fp8, x):
    q, s = fp8.quantize_fp8_rows(x.cuda())
    rq, rs = U.quantize_rows(x.float())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.float().cpu().double(), rq)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_magnitude(fp8, dtype):
    """Blocks whose largest value is at every power of two, subnormal scales and codes among them."""
    k = 128
    x = torch.randn(280, k, generator=gen(1))
    x = x * torch.exp2(torch.arange(-149, 131).float()[:, None].clamp(max=124))
    same(fp8, x.to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_borders(fp8, dtype):
    """Quotients on and beside the borders between codes: the largest value is 448 times a scale with few or many
    significant bits, the others are borders (odd multiples of half a step) times it, moved by an ulp either way."""
    steps = torch.tensor([m * 2.0 ** e for e in range(-10, 9) for m in (1.0, 1.0625, 1.1875, 1.3125, 1.4375, 1.9375)])
    steps = steps[steps < 440][:107]
    rows = []
    for s in (1.0, 0.75, 1.0078125, 3.0 ** 0.5, 1 + 2.0 ** -20, 1.875 + 2.0 ** -22, 2 - 2.0 ** -23):
        v = (steps * s).to(dtype).float()
        for move in (0, 1, -1):
            r = v.view(torch.int32) + move * (1 if dtype == F32 else 1 << 16)
            rows.append(torch.cat([torch.tensor([448.0 * s, -448.0 * s]), r.view(F32), -r.view(F32)]))
    same(fp8, torch.stack(rows).to(dtype))


def test_many_values(fp8):
    for seed in range(3):
        x = torch.randn(4000, 1024, generator=gen(seed)) * torch.rand(4000, 1, generator=gen(seed + 9)) * 30
        q, s = fp8.quantize_fp8_rows(x.to(BF16).cuda())
        p = x.to(BF16).cuda().float().unflatten(1, (8, 128))
        scale = (p.abs().amax(2).double() / U.TOP).float()
        want = (p.double() / scale[..., None]).float().to(torch.float8_e4m3fn)  # no quotient is above 448
        assert torch.equal(s, scale)
        assert torch.equal(q.float(), want.float().flatten(1))


def test_zeros_and_not_finite(fp8):
    x = torch.randn(6, 256, generator=gen(5))
    x[0] = 0
    x[1, :128] = -0.0
    x[2, 5], x[3, 200], x[4, 130] = float("inf"), float("nan"), -float("inf")
    q, s = fp8.quantize_fp8_rows(x.cuda())
    assert bool((q[0].float() == 0).all()) and bool((s[0] == 0).all()) and bool((q[1, :128].float() == 0).all())
    assert torch.isinf(s[2, 0]) and torch.isnan(s[3, 1]) and torch.isinf(s[4, 1])
    rq, rs = U.quantize_rows(x[5:6])
    assert torch.equal(q[5:6].float().cpu().double(), rq) and torch.equal(s[5:6].cpu(), rs)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [520, 384, 1001])
def test_grouped_wide_tiles(fp8, n, dtype):
    """Enough tiles for the kernel of 128 x 256: groups that end inside a tile, an odd number of column blocks, rows in
    front of the first group and behind the last, rows of y that are not whole 16 bytes."""
    k, G = 144, 40
    counts = torch.randint(0, 160, (G,), generator=gen(6)).tolist()
    counts[3], counts[7], counts[8] = 0, 300, 1
    off = [5]
    for c in counts:
        off.append(off[-1] + c)
    m = off[-1] + 9
    xq, xs = U.quantize_rows(activations(m, k, 8))
    kinds = [weights(n, k, 20 + g) for g in range(5)]
    of = [g % 5 for g in range(G)]
    wq = torch.stack([codes(kinds[g][0]).view(torch.uint8) for g in of]).view(torch.float8_e4m3fn)
    ws = torch.stack([kinds[g][1] for g in of]).cuda()
    y = torch.full((m, n), 3.0, dtype=dtype, device="cuda")
    fp8.grouped_gemm_fp8(codes(xq), xs.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), wq, ws, y)
    values = [U.values_weight(*kind) for kind in kinds]
    ref, bound = grouped_reference(xq, xs, off, [values[g] for g in of], k)
    U.assert_within(y[5: off[-1]], ref[5: off[-1]], bound[5: off[-1]], dtype)
    assert bool((y[:5] == 3.0).all()) and bool((y[off[-1]:] == 3.0).all())
