"""Products of many blocks of K in the larger tiles against 64-bit sums (on the GPU, of the values that the codes stand for);
refusals of outputs of other shapes; the layer's clusters of 4 against those of 8."""
import pytest
import torch

from tests import fp8_util as U
from tests import test_gpu_fp8_moe as moe
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


def test_outputs_of_other_shapes_are_refused(fp8):  # noqa: F811
    xq, xs, _ = operand(5, 144, 5, 20)
    wq, ws, _ = operand(40, 144, 1, 22)
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    x = torch.zeros(5, 144, dtype=BF16, device="cuda")
    for y in (torch.empty((), device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, 40, 1, device="cuda"),
              torch.empty(40, 5, device="cuda").t(), torch.empty(1, 40, device="cuda").expand(5, 40)):
        for call in (lambda: fp8.gemm_fp8(xq, xs, wq, ws, y), lambda: fp8.linear_fp8(x, wq, ws, y),
                     lambda: fp8.grouped_gemm_fp8(xq, xs, off, wq[None], ws[None], y)):
            with pytest.raises(ValueError):
                call()


def test_layer_in_clusters_of_four_and_of_eight(fp8):  # noqa: F811
    """64 tokens on 60 experts run in clusters of 4 CTAs, a few of them in clusters of 8: the same bits."""
    c = moe.Case(512, 288, 416, 60, 4, seed=30)
    layer, x = c.layer(fp8), c.x(64).cuda()
    whole = layer.forward(x)
    for a, b in ((0, 1), (3, 11), (50, 64)):
        assert torch.equal(layer.forward(x[a:b]), whole[a:b])
