"""Calls that the documentation allows and a program makes now and then: outputs that are only aligned to their elements,
the same tensor twice, wide outputs of few rows, views of larger buffers, a broadcast gate, the largest layer."""
import pytest
import torch

from tests import fp8_util as U
from tests import test_gpu_fp8_moe as moe
from tests.test_gpu_fp8 import activations, codes, fp8, gen, weights  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def shifted(rows, cols, dtype):
    """A contiguous [rows, cols] tensor one element into its buffer, and the buffer."""
    buf = torch.full((rows * cols + 9,), -5.0, dtype=dtype, device="cuda")
    return buf[1:1 + rows * cols].view(rows, cols), buf


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(3, 136, 256), (40, 200, 1040), (100, 264, 272), (300, 5000, 144)])
def test_products_into_a_shifted_output(fp8, m, n, k, dtype):
    x, (wq, ws) = activations(m, k, 1).to(BF16).cuda(), weights(n, k, 2)
    wq, ws = codes(wq), ws.cuda()
    want = fp8.linear_fp8(x, wq, ws, out_dtype=dtype)
    y, buf = shifted(m, n, dtype)
    fp8.linear_fp8(x, wq, ws, y)
    assert torch.equal(y, want)
    y.fill_(-5.0)
    assert bool((buf == -5.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [2, 30])
def test_layer_into_a_shifted_output(fp8, T, dtype):
    c = moe.Case(160, 64, 96, 7, 2, seed=11)
    layer, x = c.layer(fp8), c.x(T).cuda()
    y, buf = shifted(T, 160, dtype)
    layer.forward(x, y)
    assert torch.equal(y, layer.forward(x, out_dtype=dtype))
    y.fill_(-5.0)
    assert bool((buf == -5.0).all())


@pytest.mark.parametrize("m", [65, 128, 129, 255])
def test_wide_outputs_of_few_rows(fp8, m):
    """More column tiles than SMs."""
    n, k = 40_000, 80
    x = activations(m, k, 3).to(BF16)
    wq, ws = torch.randn(n, k, generator=gen(4)).to(torch.float8_e4m3fn), torch.rand(-(-n // 128), 1, generator=gen(5))
    y = fp8.linear_fp8(x.cuda(), wq.cuda(), ws.cuda(), out_dtype=F32)
    a, w = U.values_rows(*U.quantize_rows(x.float())), U.values_weight(wq.float(), ws)
    U.assert_within(y, a @ w.t(), U.product_bound(a, w, k), F32)


def test_one_tensor_twice(fp8):
    """Codes times themselves: the same tensor as both operands."""
    xq, xs = U.quantize_blocks(torch.randn(256, 256, generator=gen(6)))
    q, s = codes(xq), xs.cuda()
    rows = xs.repeat_interleave(128, 0).contiguous()
    y = fp8.gemm_fp8(q, rows.cuda(), q, s, out_dtype=F32)
    a, w = U.values_rows(xq, rows), U.values_weight(xq, xs)
    U.assert_within(y, a @ w.t(), U.product_bound(a, w, 256), F32)


def test_every_choice_of_an_expert(fp8):
    """All tokens on the same experts, and as many experts as choices: 64 tokens x 8 of 8."""
    c = moe.Case(96, 32, 288, 8, 8, gating=1, seed=12)
    x = c.x(64)
    c.check(x, *moe.forward(c.layer(fp8), c, x, out_dtype=F32))


def test_largest_layer(fp8):
    """d_model 8192, hidden 4096: the operands take most of an SM's shared memory.  Each row is the same bits alone and
    among others, and the first is checked."""
    c = moe.Case(8192, 4096, 4096, 2, 1, seed=13)
    layer, x = c.layer(fp8), c.x(20)
    y, idx, gate, counts = moe.forward(layer, c, x)
    assert torch.equal(layer.forward(x[19:20].cuda()), y[19:20])
    c.check(x[:1], y[:1], idx[:1], gate[:1])
    assert int(counts[:2].sum()) == 20


def test_wide_shared_expert_in_many_parts(fp8):
    c = moe.Case(64, 32, 1056, 4, 1, seed=14)
    x = c.x(19)
    c.check(x, *moe.forward(c.layer(fp8), c, x))


@pytest.mark.parametrize("n", [40, 1200])
def test_many_groups(fp8, n):
    """1024 groups, most of them empty or of a row or two, a few offsets that go back; each a small product of its own."""
    k, G = 16, 1024
    counts = torch.randint(0, 4, (G,), generator=gen(15)) * (torch.rand(G, generator=gen(16)) < 0.4)
    counts[100:300] = 0
    counts[511], counts[512], counts[1023] = 140, 0, 5
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    m = int(off[-1])
    given = off.clone()
    given[150], given[200], given[250] = 0, -9, 3  # inside an empty stretch: taken as what is before them
    xq, xs = U.quantize_rows(activations(m, k, 17))
    wq = torch.randn(G, n, k, generator=gen(18)).to(torch.float8_e4m3fn)
    ws = torch.rand(G, -(-n // 128), 1, generator=gen(19))
    y = fp8.grouped_gemm_fp8(codes(xq), xs.cuda(), given.int().cuda(), wq.cuda(), ws.cuda(), out_dtype=F32)
    a = U.values_rows(xq, xs)
    of = torch.searchsorted(off[1:], torch.arange(m), right=True)
    w = wq.double() * ws.double().repeat_interleave(128, 1)[:, :n]
    ref = torch.einsum("mk,mnk->mn", a, w[of])
    size = torch.einsum("mk,mnk->mn", a.abs(), w[of].abs())
    U.assert_within(y, ref, size * (128 * 2 + 11) * 2.0 ** -24 + 2.0 ** -120, F32)
