"""Products of many blocks of K in the larger tiles against 64-bit sums (on the GPU, of the values that the codes stand for)."""
import pytest
import torch

from tests import fp8_util as U
from tests.test_gpu_fp8 import fp8, gen  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def operand(rows, k, scale_rows, seed):
    """Random codes and scales (one a row or one a 128 rows) and what they stand for."""
    q = torch.randn(rows, k, generator=gen(seed)).mul_(60).to(torch.float8_e4m3fn).cuda()
    s = (0.01 + torch.rand(scale_rows, U.blocks(k), generator=gen(seed + 1))).cuda()
    each = s if scale_rows == rows else s.repeat_interleave(U.BLOCK, 0)[:rows]
    return q, s, q.double() * each.double().repeat_interleave(U.BLOCK, 1)[:, :k]


# pairs of CTAs (more and fewer tiles than pairs, rows and columns that end inside a tile), one tile of rows with many
# columns (128 x 256), and tiles of 128 x 128 for comparison
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(5000, 1100, 2064), (9000, 512, 4240), (2100, 2304, 1024), (20000, 264, 1296),
                                   (100, 38000, 784), (700, 640, 4240)])
def test_deep_products(fp8, m, n, k, dtype):  # noqa: F811
    xq, xs, a = operand(m, k, m, 1)
    wq, ws, w = operand(n, k, U.blocks(n), 3)
    y = fp8.gemm_fp8(xq, xs, wq, ws, out_dtype=dtype)
    U.assert_within(y, (a @ w.t()).cpu(), U.product_bound(a, w, k).cpu(), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_deep_groups(fp8, dtype):  # noqa: F811
    """Tiles of 128 x 256 over 17 blocks of K, groups of 0 to 400 rows."""
    counts, n, k = [400, 0, 129, 1, 128, 255, 77, 300] * 4, 1048, 2064
    off = torch.tensor([0, *counts]).cumsum(0)
    m, groups = int(off[-1]), len(counts)
    xq, xs, a = operand(m, k, m, 5)
    parts = [operand(n, k, U.blocks(n), 7 + 2 * g) for g in range(groups)]
    wq = torch.stack([q.view(torch.uint8) for q, _, _ in parts]).view(torch.float8_e4m3fn)
    y = fp8.grouped_gemm_fp8(xq, xs, off.int().cuda(), wq, torch.stack([s for _, s, _ in parts]), out_dtype=dtype)
    for g, (_, _, w) in enumerate(parts):
        rows = slice(int(off[g]), int(off[g + 1]))
        U.assert_within(y[rows], (a[rows] @ w.t()).cpu(), U.product_bound(a[rows], w, k).cpu(), dtype)
