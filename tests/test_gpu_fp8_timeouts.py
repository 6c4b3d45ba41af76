"""Bounded waits of the e4m3 products and the layer that run out, without a GPU fault: barriers that expect an arrival more
than there is, under a limit of microseconds.  The kernel drains what it has in flight and returns, the context stays usable, the timeout is
reported once, and the next call is right again."""
import pytest
import torch

from moe_ffn_layer_fp32_b200 import _lib
from tests.test_gpu_fp8 import codes, fp8, gen, weights  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TIMEOUT = 5


@pytest.fixture(autouse=True)
def default_waits(fp8):  # noqa: F811
    yield
    torch.cuda.synchronize()
    assert _lib.lib().mmoe_debug_fp8_waits(0, 0) == 0
    _lib.lib().mmoe_fp8_status()


def waits(clocks, stall=0):
    assert _lib.lib().mmoe_debug_fp8_waits(clocks, stall) == 0


def linear(fp8, m, n, k):
    x = torch.randn(m, k, generator=gen(1)).to(BF16).cuda()
    wq = torch.randn(n, k, generator=gen(2)).to(torch.float8_e4m3fn).cuda()
    ws = torch.rand(-(-n // 128), -(-k // 128), generator=gen(3)).cuda()
    return lambda: fp8.linear_fp8(x, wq, ws, out_dtype=F32)


def grouped(fp8, m, groups, n, k):
    xq = torch.randn(m, k, generator=gen(4)).to(torch.float8_e4m3fn).cuda()
    xs = torch.rand(m, -(-k // 128), generator=gen(5)).cuda()
    wq = torch.randn(groups, n, k, generator=gen(6)).to(torch.float8_e4m3fn).cuda()
    ws = torch.rand(groups, -(-n // 128), -(-k // 128), generator=gen(7)).cuda()
    off = (torch.arange(groups + 1) * m // groups).int().cuda()
    return lambda: fp8.grouped_gemm_fp8(xq, xs, off, wq, ws, out_dtype=F32)


def layer(fp8, T, d, h, hs, E, k):
    def codes_of(*shape):
        return (0.5 * torch.randn(shape, generator=gen(8))).to(torch.float8_e4m3fn).cuda()

    def scales(*shape):
        return 0.1 * torch.rand(shape, generator=gen(9)).cuda()

    def b(n):
        return -(-n // 128)
    moe = fp8.FP8MoELayer(d, h, shared_hidden=hs, n_experts=E, top_k=k)
    moe.load(0.05 * torch.randn(d, E, generator=gen(10)).cuda(), None, codes_of(E, 2 * h, d), scales(E, 2 * b(h), b(d)),
             codes_of(E, d, h), scales(E, b(d), b(h)), codes_of(2 * hs, d), scales(2 * b(hs), b(d)), codes_of(d, hs),
             scales(b(d), b(hs)))
    x = torch.randn(T, d, generator=gen(11)).to(BF16).cuda()
    return lambda: moe.forward(x)


# every kernel: few rows with 16, 32 and 64 operand rows, a cluster or one CTA along K, one round of K or several; tiles
# of 128 x 128 and 128 x 256 and pairs of CTAs, several tiles a CTA; the layer in clusters of 8 and of 4
CALLS = {"few rows, 8 CTAs": (linear, 3, 256, 2048), "few rows, one CTA": (linear, 20, 12000, 256),
         "few rows, rounds": (linear, 64, 200, 12288), "small tiles": (linear, 777, 1000, 784),
         "pairs": (linear, 12000, 1024, 1024), "pairs of one block": (linear, 6000, 1024, 128),
         "groups, wide tiles": (grouped, 900, 40, 1024, 528), "groups, small tiles": (grouped, 200, 3, 264, 144),
         "layer, 1 token": (layer, 1, 512, 256, 256, 12, 4), "layer, 8 tokens": (layer, 8, 768, 384, 1536, 60, 4),
         "layer, 64 tokens": (layer, 64, 1024, 256, 256, 60, 4), "layer, few features": (layer, 9, 64, 32, 160, 4, 2)}


@pytest.fixture(scope="module", params=list(CALLS))
def call(request, fp8):  # noqa: F811
    make, *sizes = CALLS[request.param]
    run = make(fp8, *sizes)
    return run, run().clone()


@pytest.mark.parametrize("stall", [1, 2])
def test_a_stall_is_reported_by_the_next_call(fp8, call, stall):  # noqa: F811
    run, want = call
    waits(40_000, stall)                # about 20 us
    run()                               # enqueues: the stall happens on the device
    torch.cuda.synchronize()            # the context is still usable
    waits(0)
    with pytest.raises(_lib.MMoEError) as error:
        run()
    assert error.value.status == TIMEOUT
    assert torch.equal(run(), want)     # reported once, and right again
    fp8.check_timeouts()


@pytest.mark.parametrize("stall", [1, 2])
def test_a_stall_is_reported_by_the_status(fp8, call, stall):  # noqa: F811
    run, want = call
    waits(40_000, stall)
    run()
    torch.cuda.synchronize()
    waits(0)
    with pytest.raises(_lib.MMoEError) as error:
        fp8.check_timeouts()
    assert error.value.status == TIMEOUT
    fp8.check_timeouts(torch.device("cuda", torch.cuda.current_device()))
    assert torch.equal(run(), want)


def test_a_short_limit_never_gives_a_wrong_result_as_right(fp8, call):  # noqa: F811
    """Every wait may give up at once, wherever the kernel stands."""
    run, want = call
    for _ in range(8):
        waits(1)
        y = run()
        torch.cuda.synchronize()
        waits(0)
        try:
            fp8.check_timeouts()
        except _lib.MMoEError as error:
            assert error.status == TIMEOUT
        else:
            assert torch.equal(y, want)
        assert torch.equal(run(), want)


def test_replays_are_reported_by_the_status(fp8):  # noqa: F811
    """A captured call keeps its stall, so that each replay runs out; no call reports that, the status does."""
    run = linear(fp8, 40, 512, 1024)
    want = run().clone()
    graph = torch.cuda.CUDAGraph()
    waits(40_000, 1)
    with torch.cuda.graph(graph):
        run()
    waits(0)
    fp8.check_timeouts()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        with pytest.raises(_lib.MMoEError):
            fp8.check_timeouts()
        fp8.check_timeouts()
    assert torch.equal(run(), want)
