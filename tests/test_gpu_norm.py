"""The block norm on the GPU against a plain 64-bit form."""
import pytest
import torch

from tests import fp8_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# A thread adds at most 32 squares in a row, then come 5 + 3 levels of partial sums, the mean, eps, the root, the
# quotient and the products with it: no more than 64 roundings on any path from an input to an output.
U64 = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def norm():
    from moe_ffn_layer_fp32_b200 import build
    from moe_ffn_layer_fp32_b200.norm import block_norm
    build.build()
    return block_norm


def gen(seed):
    return torch.Generator().manual_seed(seed)


def reference(r, y, post, gate, scale, pre, eps):
    """r', x in 64 bits and how far FP32 may be off."""
    r = r.double()
    if y is None:
        z = torch.zeros_like(r)
    else:
        z = y.double()
        if post is not None:
            z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * post.double()
        if gate is not None:
            z = z * gate.double()
    out = scale * r + z
    off = U64 * (z.abs() + out.abs() + (scale * r).abs())
    if pre is None:
        return out, off, None, None
    ms = out.square().mean(-1, keepdim=True) + eps
    x = out / ms.sqrt() * pre.double()
    moved = (out.abs() * off).mean(-1, keepdim=True) / ms  # relative change of the root mean square
    return out, off, x, pre.double().abs() * off / ms.sqrt() + x.abs() * (moved + U64)


def check(got, want, quantize):
    r, x, xq, sx = got
    rr, roff, xr, xoff = want
    if r is not None:
        U.assert_within(r, rr, roff, r.dtype)
    if xr is None:
        assert x is None and xq is None and sx is None
        return
    U.assert_within(x, xr, xoff, BF16)
    if not quantize:
        assert xq is None and sx is None
        return
    # each code stands for its value to within half a step: 2^-4 of it, or half of the smallest step 2^-9
    s = sx.double().cpu().repeat_interleave(U.BLOCK, 1)[:, : xr.shape[1]]
    half = (xr.abs() + xoff) * 2.0 ** -4
    half = torch.maximum(half, s * 2.0 ** -10)
    U.assert_within(xq.float().double().cpu() * s, xr, half + xoff, F32)
    for b in range(sx.shape[1]):
        at = slice(b * U.BLOCK, (b + 1) * U.BLOCK)
        top, o = xr[:, at].abs().amax(1), xoff[:, at].amax(1)
        assert bool(((sx[:, b].double().cpu() * U.TOP - top).abs() <= o + top * 2.0 ** -23).all())


GATES = {"none": lambda t, d: None, "channel": lambda t, d: torch.rand(d, generator=gen(4)),
         "token": lambda t, d: torch.rand(t, 1, generator=gen(4)), "full": lambda t, d: torch.rand(t, d, generator=gen(4))}


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("rt,yt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("t,d", [(1, 8), (3, 256), (17, 264), (33, 512), (5, 768), (9, 1032), (2, 2048), (7, 2056), (3, 4104),
                                 (2, 8192)])
def test_whole(norm, t, d, rt, yt, gate, quantize):
    r, y = 3 * torch.randn(t, d, generator=gen(1)), torch.randn(t, d, generator=gen(2))
    r, y = r.to(rt), y.to(yt)
    post, pre = torch.randn(d, generator=gen(3)), torch.randn(d, generator=gen(5))
    g = GATES[gate](t, d)
    got = norm(r.cuda(), y.cuda(), post_weight=post.cuda(), gate=None if g is None else g.cuda(), residual_scale=0.75,
               pre_weight=pre.cuda(), eps=1e-5, quantize=quantize)
    check(got, reference(r, y, post, g, 0.75, pre, 1e-5), quantize)


@pytest.mark.parametrize("t,d", [(5, 264), (300, 2048)])
def test_parts(norm, t, d):
    r, y = torch.randn(t, d, generator=gen(6)).to(BF16), torch.randn(t, d, generator=gen(7))
    w = torch.rand(d, generator=gen(8))
    check(norm(r.cuda(), y.cuda()), reference(r, y, None, None, 1.0, None, 1e-6), False)
    check(norm(r.cuda(), y.cuda(), pre_weight=w.cuda()), reference(r, y, None, None, 1.0, w, 1e-6), False)
    check(norm(r.cuda(), y.cuda(), post_weight=w.cuda(), residual_scale=0.0), reference(r, y, w, None, 0.0, None, 1e-6), False)
    got = norm(r.cuda(), pre_weight=w.cuda(), quantize=True)
    assert got[0] is None
    check(got, reference(r, None, None, None, 1.0, w, 1e-6), True)
    held = torch.empty(t, d, dtype=BF16, device="cuda")
    assert norm(r.cuda(), residual_scale=2.0, out_residual=held)[0] is held
    assert torch.equal(held.cpu(), r * 2)


def test_zero_rows_and_not_finite_rows(norm):
    """A row of zeros (eps keeps it finite), one of subnormals, and a NaN and infinities that stay in their rows."""
    t, d = 8, 512
    r, y = torch.randn(t, d, generator=gen(9)), torch.randn(t, d, generator=gen(10))
    w = torch.ones(d)
    r[0], y[0] = 0, 0
    y[1] *= 1e-40
    want = reference(r, y, w, None, 1.0, w, 1e-6)
    check(norm(r.cuda(), y.cuda(), post_weight=w.cuda(), pre_weight=w.cuda(), quantize=True), want, True)
    clean = norm(r.cuda(), y.cuda(), post_weight=w.cuda(), pre_weight=w.cuda(), quantize=True)
    r[3, 7], y[5, 300] = float("inf"), float("nan")
    got = norm(r.cuda(), y.cuda(), post_weight=w.cuda(), pre_weight=w.cuda(), quantize=True)
    assert torch.isnan(got[0][5]).all() and torch.isnan(got[1][5]).all() and torch.isnan(got[3][5]).all()
    assert torch.isinf(got[0][3, 7]) and torch.isnan(got[1][3, 7])
    keep = [0, 1, 2, 4, 6, 7]
    for a, b in zip(got, clean):
        assert torch.equal(a.view(torch.uint8)[keep], b.view(torch.uint8)[keep])


def test_strided_in_place_and_frames(norm):
    t, d = 37, 520
    big = torch.randn(t, d + 24, generator=gen(11)).cuda()
    r0 = big[:, 8:8 + d].clone()
    y = torch.randn(t, d + 8, generator=gen(12)).to(BF16).cuda()[:, :d]
    gate = torch.rand(t, d + 4, generator=gen(13)).cuda()[:, :d]
    w = torch.rand(d, generator=gen(14)).cuda()
    want = norm(r0, y, post_weight=w, gate=gate, pre_weight=w)
    frame = big.clone()
    view = frame[:, 8:8 + d]
    got = norm(view, y, post_weight=w, gate=gate, pre_weight=w, out_residual=view)
    assert torch.equal(view, want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(frame[:, :8], big[:, :8]) and torch.equal(frame[:, 8 + d:], big[:, 8 + d:])
    # a gate with broadcast rows
    row = torch.rand(1, d, generator=gen(15)).cuda()
    assert torch.equal(norm(r0, y, gate=row)[0], norm(r0, y, gate=row.expand(t, d))[0])
    assert torch.equal(norm(r0, y, gate=row)[0], norm(r0, y, gate=row[0])[0])


def test_no_rows_captured_and_other_stream(norm):
    d = 1024
    w = torch.rand(d, generator=gen(16)).cuda()
    none = norm(torch.empty(0, d, device="cuda"), torch.empty(0, d, device="cuda"), pre_weight=w, quantize=True)
    assert [tuple(v.shape) for v in none] == [(0, d), (0, d), (0, d), (0, 8)]
    r, y = torch.randn(50, d, generator=gen(17)).cuda(), torch.randn(50, d, generator=gen(18)).cuda()
    want = norm(r, y, pre_weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm(r, y, pre_weight=w, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = norm(r, y, pre_weight=w, quantize=True)
    r.mul_(-0.5)
    graph.replay()
    for a, b in zip(held, norm(r, y, pre_weight=w, quantize=True)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_codes_feed_the_product(norm):
    """x's codes and scales are what the e4m3 product takes."""
    from moe_ffn_layer_fp32_b200 import fp8
    t, d, n = 90, 272, 200
    r = torch.randn(t, d, generator=gen(19))
    wq, ws = U.quantize_blocks(0.02 * torch.randn(n, d, generator=gen(20)))
    _, _, xq, sx = norm(r.cuda(), pre_weight=torch.ones(d).cuda(), quantize=True)
    y = fp8.gemm_fp8(xq, sx, wq.float().to(torch.float8_e4m3fn).cuda(), ws.cuda(), out_dtype=F32)
    a, w = U.values_rows(xq.float().cpu(), sx.cpu()), U.values_weight(wq, ws)
    U.assert_within(y, a @ w.t(), U.product_bound(a, w, d), F32)


def test_offsets_past_32_bits(norm):
    t, d = 300_000, 8192
    r = torch.empty(t, d, dtype=BF16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    w = torch.rand(d, generator=gen(21)).cuda()
    _, x, xq, sx = norm(r, pre_weight=w, quantize=True)
    for at in (0, 262_100, t - 64):
        want = norm(r[at:at + 64], pre_weight=w, quantize=True)
        for a, b in zip((x, xq, sx), want[1:]):
            assert torch.equal(a[at:at + 64].view(torch.uint8), b.view(torch.uint8))
