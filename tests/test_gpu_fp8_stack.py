"""The e4m3 operators and the block norm together, as a decoder's blocks use them: norm, MoE layer, norm with codes, a
projection on the codes.  Each step is checked on the inputs that it had on the GPU; the whole runs eagerly, on another
stream and as a captured graph with the same bits."""
import numpy as np
import pytest
import torch

from tests import fp8_util as U
from tests import test_gpu_fp8_moe as moe
from tests import test_gpu_norm as norms

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from moe_ffn_layer_fp32_b200 import build, fp8
    from moe_ffn_layer_fp32_b200.norm import block_norm
    build.build()
    return fp8, block_norm


def step(fp8, block_norm, layers, params, w, r, stream=None):
    """The residual stream and everything in between, of a stack of blocks."""
    seen = []
    _, x, _, _ = block_norm(r, pre_weight=params[0]["pre"], stream=stream)
    for layer, p in zip(layers, params):
        y = layer.forward(x, stream=stream)
        r2, x2, xq, sx = block_norm(r, y, post_weight=p["post"], gate=p["gate"], residual_scale=0.875, pre_weight=p["next"],
                                    quantize=True, stream=stream)
        z = fp8.gemm_fp8(xq, sx, *w, out_dtype=F32, stream=stream)
        seen.append((r, x, y, r2, x2, xq, sx, z))
        r, x = r2, x2
    return seen


def parameters(d, n, seed):
    out = []
    for i in range(n):
        g = moe.gen(seed + i)
        out.append({k: 1 + 0.1 * torch.randn(d, generator=g) for k in ("pre", "post", "gate", "next")})
    return out


@pytest.mark.parametrize("T", [1, 7, 64])
def test_fp8_stack(ops, T):
    fp8, block_norm = ops
    d = 192
    cases = [moe.Case(d, 96, 160, 9, 3, gating=i % 3, bias=i == 2, seed=50 * i) for i in range(3)]
    layers = [c.layer(fp8) for c in cases]
    params = parameters(d, 3, 7)
    on = [{k: v.cuda() for k, v in p.items()} for p in params]
    wq, ws = U.quantize_blocks(0.02 * torch.randn(200, d, generator=moe.gen(1)))
    w = (wq.float().to(torch.float8_e4m3fn).cuda(), ws.cuda())
    r = (2 * torch.randn(T, d, generator=moe.gen(2))).to(BF16).cuda()
    seen = step(fp8, block_norm, layers, on, w, r)
    for c, p, (r0, x, y, r2, x2, xq, sx, z) in zip(cases, params, seen):
        xc = x.cpu()
        idx, gate, counts = moe.outputs(c, T)
        again = c.layer(fp8).forward(x, topk_idx=idx, topk_gate=gate, expert_counts=counts)
        assert torch.equal(again, y)
        c.check(xc, y, idx.cpu(), gate.cpu(), counts.cpu())
        norms.check((r2, x2, xq, sx), norms.reference(r0.cpu(), y.cpu(), p["post"], p["gate"], 0.875, p["next"], 1e-6), True)
        a, b = U.values_rows(xq.float().cpu(), sx.cpu()), U.values_weight(wq, ws)
        U.assert_within(z, a @ b.t(), U.product_bound(a, b, d), F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(fp8, block_norm, layers, on, w, r, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(fp8, block_norm, layers, on, w, r)
    for _ in range(3):
        graph.replay()
    for a, b, c in zip(seen, other, held):
        for u, v, h in zip(a, b, c):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)) and torch.equal(u.view(torch.uint8), h.view(torch.uint8))


def test_norm_between_int4_layers(ops, c0_layer):
    """The norm's BF16 rows are what the INT4 layer takes, its FP32 rows what the norm takes; one captured graph."""
    import oracle
    from moe_ffn_layer_fp32_b200.layer import MoELayer
    _, block_norm = ops
    _, _, q, x = c0_layer
    layer = MoELayer(q.d, q.h, shared_hidden=q.hs, max_tokens=x.shape[0], decode=True, deterministic=True, device=0)
    layer.load(q.w_router, q.router_bias, q.w_gate_up, q.s_gate_up, q.w_down, q.s_down)
    p = {k: v.cuda() for k, v in parameters(q.d, 1, 3)[0].items()}
    r = torch.from_numpy(x.view(np.int16)).cuda().view(BF16)

    def run():
        _, a, _, _ = block_norm(r, pre_weight=p["pre"])
        y = layer.forward(a)
        return a, y, *block_norm(r, y, post_weight=p["post"], gate=p["gate"], pre_weight=p["next"])[:2]

    a, y, r2, x2 = run()
    want = oracle.moe_layer(q, a.view(torch.int16).cpu().numpy().view(x.dtype))
    want = want[0] if isinstance(want, tuple) else want
    assert float(np.abs(y.cpu().numpy() - want).max()) <= 2e-3 * float(np.abs(want).max())
    host = {k: v.cpu() for k, v in p.items()}
    norms.check((r2, x2, None, None), norms.reference(r.cpu(), y.cpu(), host["post"], host["gate"], 1.0, host["next"], 1e-6), False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    graph.replay()
    for u, v in zip((a, y, r2, x2), held):
        assert torch.equal(u, v)
    layer.close()
