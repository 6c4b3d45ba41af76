"""The e4m3 quantisers and products on the GPU against plain 64-bit forms."""
import pytest
import torch

from tests import fp8_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BLOCK = U.BLOCK


@pytest.fixture(scope="module")
def fp8():
    from moe_ffn_layer_fp32_b200 import build, fp8
    build.build()
    return fp8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activations(m, k, seed):
    """Normal values with a few large features, a zero block, a block of subnormals and one row of zeros."""
    x = torch.randn(m, k, generator=gen(seed))
    x[:, torch.randperm(k, generator=gen(seed + 1))[: max(1, k // 64)]] *= 20
    x[0, :BLOCK] = 0
    if m > 2:
        x[1, :BLOCK] *= 1e-38
        x[2] = 0
    return x



def weights(n, k, seed):
    return U.quantize_blocks(0.02 * torch.randn(n, k, generator=gen(seed)))


def codes(q):
    return q.to(F32).to(torch.float8_e4m3fn).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,k", [(1, 8), (3, 128), (5, 136), (70, 1000), (129, 2048)])
def test_quantize_rows(fp8, m, k, dtype):
    x = activations(m, k, 1).to(dtype)
    q, s = fp8.quantize_fp8_rows(x.cuda())
    rq, rs = U.quantize_rows(x.float())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.float().cpu().double(), rq)


def test_quantize_rows_strided_and_not_finite(fp8):
    x = activations(9, 400, 2).to(BF16)
    x[3, 5], x[4, 200], x[5, 399] = float("nan"), float("inf"), -float("inf")
    full = x.cuda()
    q, s = fp8.quantize_fp8_rows(full[:, 16:280])
    part = x[:, 16:280].float()
    rq, rs = U.quantize_rows(part)
    assert torch.equal(s.cpu(), rs) and torch.isinf(s[4, 1])
    assert torch.equal(q.float().cpu().double().nan_to_num(7), rq.nan_to_num(7))
    q, s = fp8.quantize_fp8_rows(full)
    assert torch.isnan(s[3, 0]) and torch.isinf(s[5, 3]) and torch.isfinite(s[6]).all()


@pytest.mark.parametrize("shape", [(1, 8), (128, 128), (200, 272), (3, 130, 264), (2, 2, 16, 48)])
def test_quantize_blocks(fp8, shape):
    w = torch.randn(shape, generator=gen(3))
    w[..., : min(128, shape[-2]), : min(128, shape[-1])][..., 0, :] = 0
    for v in (w, w.to(BF16)):
        q, s = fp8.quantize_fp8_blocks(v.cuda())
        for i, one in enumerate(v.float().reshape(-1, *shape[-2:])):
            rq, rs = U.quantize_blocks(one)
            assert torch.equal(s.reshape(-1, *s.shape[-2:])[i].cpu(), rs)
            assert torch.equal(q.float().cpu().double().reshape(-1, *shape[-2:])[i], rq)


# few rows on one launch (16, 32 and 64 operand rows, K in one or several rounds of the operand buffer), many rows on
# the tile kernel (one and two halves), every size ending inside its tile
SIZES = [(1, 1, 16), (1, 128, 128), (1, 2048, 1024), (16, 100, 144), (17, 129, 272), (33, 200, 5008), (64, 257, 2048),
         (64, 136, 12288), (65, 64, 16), (128, 128, 128), (130, 257, 784), (777, 1000, 400), (2500, 2050, 272),
         (19000, 264, 144)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_and_linear(fp8, m, n, k, dtype):
    x = activations(m, k, 4).to(BF16)
    (xq, xs), (wq, ws) = U.quantize_rows(x.float()), weights(n, k, 5)
    a, w = U.values_rows(xq, xs), U.values_weight(wq, ws)
    y = fp8.gemm_fp8(codes(xq), xs.cuda(), codes(wq), ws.cuda(), out_dtype=dtype)
    U.assert_within(y, a @ w.t(), U.product_bound(a, w, k), dtype)
    z = fp8.linear_fp8(x.cuda(), codes(wq), ws.cuda(), out_dtype=dtype)
    assert torch.equal(y, z)


def framed(m, n, ld, dtype, value=-7.0):
    """An [m, n] view of rows ld apart inside a buffer of sentinels, and the buffer."""
    buf = torch.full((m + 3, ld), value, dtype=dtype, device="cuda")
    return buf[1:m + 1, 8:8 + n], buf


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k,ld", [(5, 100, 144, 128), (64, 130, 256, 139), (200, 100, 144, 120), (300, 259, 272, 275)])
def test_output_rows_apart(fp8, m, n, k, ld, dtype):
    x = activations(m, k, 6).to(BF16)
    wq, ws = weights(n, k, 7)
    ref = fp8.linear_fp8(x.cuda(), codes(wq), ws.cuda(), out_dtype=dtype)
    wide = torch.zeros(m, k + 24, dtype=BF16)
    wide[:, 8:8 + k] = x
    y, buf = framed(m, n, ld, dtype)
    assert fp8.linear_fp8(wide.cuda()[:, 8:8 + k], codes(wq), ws.cuda(), y) is y
    assert torch.equal(y, ref)
    y.fill_(-7.0)
    assert bool((buf == -7.0).all()), "something outside y was written"


def grouped_reference(xq, xs, offsets, w, k):
    a = U.values_rows(xq, xs)
    ref = torch.zeros(a.shape[0], w[0].shape[0], dtype=torch.float64)
    bound = torch.zeros_like(ref)
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        ref[lo:hi] = a[lo:hi] @ w[g].t()
        bound[lo:hi] = U.product_bound(a[lo:hi], w[g], k)
    return ref, bound


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("counts,n,k", [([1], 128, 128), ([0, 5, 0, 0, 130, 1], 100, 144), ([128, 128, 256], 264, 272),
                                        ([3] * 40, 136, 400), ([0] * 33 + [2] + [0] * 40, 72, 16),
                                        ([700, 0, 90, 1300], 1160, 272)])
def test_grouped(fp8, counts, n, k, dtype):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    x = activations(off[-1] + 9, k, 8)  # nine rows behind the last group
    xq, xs = U.quantize_rows(x)
    pairs = [weights(n, k, 20 + g) for g in range(len(counts))]
    wq, ws = torch.stack([codes(q).view(torch.uint8) for q, _ in pairs]).view(torch.float8_e4m3fn), torch.stack([s for _, s in pairs])
    y = torch.full((off[-1] + 9, n), 3.0, dtype=dtype, device="cuda")
    fp8.grouped_gemm_fp8(codes(xq), xs.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), wq, ws.cuda(), y)
    ref, bound = grouped_reference(xq[: off[-1]], xs[: off[-1]], off, [U.values_weight(q, s) for q, s in pairs], k)
    U.assert_within(y[: off[-1]], ref, bound, dtype)
    assert bool((y[off[-1]:] == 3.0).all()), "rows behind the last group were written"


def test_grouped_offsets_out_of_range(fp8):
    """Offsets out of [0, M] or out of order are taken as the nearest that are not; no other row is written."""
    n, k, m = 40, 144, 50
    xq, xs = U.quantize_rows(activations(m, k, 9))
    pairs = [weights(n, k, 30 + g) for g in range(5)]
    wq, ws = torch.stack([codes(q).view(torch.uint8) for q, _ in pairs]).view(torch.float8_e4m3fn), torch.stack([s for _, s in pairs])
    for given, meant in (([-5, 10, 3, 20, 99, 7], [0, 10, 10, 20, 50, 50]), ([4, 4, 9, -1, 9, 30], [4, 4, 9, 9, 9, 30])):
        y = torch.full((m, n), 3.0, device="cuda")
        fp8.grouped_gemm_fp8(codes(xq), xs.cuda(), torch.tensor(given, dtype=torch.int32).cuda(), wq, ws.cuda(), y)
        ref, bound = grouped_reference(xq, xs, meant, [U.values_weight(q, s) for q, s in pairs], k)
        U.assert_within(y[meant[0]:meant[-1]], ref[meant[0]:meant[-1]], bound[meant[0]:meant[-1]], F32)
        assert bool((y[: meant[0]] == 3.0).all()) and bool((y[meant[-1]:] == 3.0).all())


@pytest.mark.parametrize("m", [3, 200])
def test_not_finite_rows_stay_apart(fp8, m):
    """A NaN or infinity reaches its own row's outputs and no other's."""
    k, n = 400, 150
    x = activations(m, k, 10).to(BF16)
    wq, ws = weights(n, k, 11)
    clean = fp8.linear_fp8(x.cuda(), codes(wq), ws.cuda(), out_dtype=F32)
    bad = x.clone()
    bad[0, 390], bad[2, 1] = float("nan"), float("inf")
    y = fp8.linear_fp8(bad.cuda(), codes(wq), ws.cuda(), out_dtype=F32)
    assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all()
    keep = [i for i in range(m) if i not in (0, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("m", [0, 5, 200])
def test_no_rows_captured_and_other_stream(fp8, m):
    k, n = 272, 200
    wq, ws = weights(n, k, 13)
    wq, ws = codes(wq), ws.cuda()
    x = torch.randn(m, k, generator=gen(12)).to(BF16).cuda()
    want = fp8.linear_fp8(x, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = fp8.linear_fp8(x, wq, ws, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and y.shape == (m, n)
    if m == 0:
        return
    fresh = torch.randn(m, k, generator=gen(14)).to(BF16).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fp8.linear_fp8(x, wq, ws)
    for v in (x.clone(), fresh):
        x.copy_(v)
        graph.replay()
        assert torch.equal(held, fp8.linear_fp8(v, wq, ws))


def test_two_streams_at_once(fp8):
    """Calls in flight together share nothing."""
    cases = []
    for m, n, k, seed in ((64, 2048, 2048, 15), (3000, 1024, 1024, 16)):
        wq, ws = weights(n, k, seed)
        cases.append((torch.randn(m, k, generator=gen(seed)).to(BF16).cuda(), codes(wq), ws.cuda()))
    want = [fp8.linear_fp8(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[fp8.linear_fp8(*c, stream=s) for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for y, w in zip(pair, want):
            assert torch.equal(y, w)


def test_offsets_past_32_bits(fp8):
    """More than 2^31 output elements: the last rows are those of a small product."""
    m, n, k = 560_000, 4096, 16
    x = torch.randn(m, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    wq, ws = weights(n, k, 17)
    wq, ws = codes(wq), ws.cuda()
    y = fp8.linear_fp8(x, wq, ws)
    for at in (0, 524_200, m - 200):
        assert torch.equal(y[at:at + 200], fp8.linear_fp8(x[at:at + 200], wq, ws))
