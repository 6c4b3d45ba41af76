"""The MoE layer on e4m3 weights for up to 64 tokens against a 64-bit form, element by element.

The bound follows the formula.  Where an FP32 sum may leave a hidden feature between two codes, both codes are allowed:
the code lies between those of the smallest and the largest ratio that the bounds of the steps before admit."""
import pytest
import torch

from tests import fp8_util as U

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
BLOCK = U.BLOCK
H = 2.0 ** -24  # half a step of FP32, relative


@pytest.fixture(scope="module")
def fp8():
    from moe_ffn_layer_fp32_b200 import build, fp8
    build.build()
    return fp8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weight(n, k, seed):
    return U.quantize_blocks(0.04 * torch.randn(n, k, generator=gen(seed)))


class Case:
    """A layer's weights, quantised here, and what they stand for in 64 bits."""

    def __init__(self, d, h, hs, E, k, gating=0, bias=False, seed=0):
        self.d, self.h, self.hs, self.E, self.k, self.gating = d, h, hs, E, k, gating
        self.router = 0.05 * torch.randn(d, E, generator=gen(seed))
        self.bias = 0.1 * torch.randn(E, generator=gen(seed + 1)) if bias else None
        # at most 12 different experts (the CPU quantises slowly), dealt out in turn
        self.kinds = [self.expert(h, seed + 10 + 3 * i) for i in range(min(E, 12))]
        self.shared = self.expert(hs, seed + 5)

    def expert(self, h, seed):
        return weight(h, self.d, seed), weight(h, self.d, seed + 1), weight(self.d, h, seed + 2)

    def ffn_of(self, e):
        return self.shared if e == self.E else self.kinds[e % len(self.kinds)]

    @staticmethod
    def packed(experts):
        def code(q):
            return q.float().to(torch.float8_e4m3fn).view(torch.uint8)
        gu = torch.stack([torch.cat([code(g[0]), code(u[0])]) for g, u, _ in experts])
        sgu = torch.stack([torch.cat([g[1], u[1]]) for g, u, _ in experts])
        dn = torch.stack([code(w[0]) for _, _, w in experts])
        return [t.cuda() for t in (gu.view(torch.float8_e4m3fn), sgu, dn.view(torch.float8_e4m3fn),
                                   torch.stack([w[1] for _, _, w in experts]))]

    def layer(self, fp8, max_tokens=64):
        out = fp8.FP8MoELayer(self.d, self.h, shared_hidden=self.hs, n_experts=self.E, top_k=self.k, gating=self.gating,
                              has_router_bias=self.bias is not None, max_tokens=max_tokens)
        of = torch.arange(self.E, device="cuda") % len(self.kinds)
        routed = [t.view(torch.uint8)[of].view(t.dtype) if t.dtype != F32 else t[of] for t in self.packed(self.kinds)]
        shared = [t[0] for t in self.packed([self.shared])]
        out.load(self.router.cuda(), None if self.bias is None else self.bias.cuda(), *routed, *shared)
        return out

    def x(self, T, seed=99):
        x = torch.randn(T, self.d, generator=gen(seed))
        x[:, :: 61] *= 9
        return x.to(BF16)

    # ---- the formula in 64 bits, with bounds

    def keys(self, x):
        """Selection keys, scores (before the normalisation of the k selected) and the bound of the keys."""
        x = x.double()
        w = self.router.double()
        logit = x @ w
        # a sum of d products in FP32, in whatever order: each term passes fewer than d + 16 roundings
        err = (self.d + 16) * H * (x.abs() @ w.abs())
        b = 0.0 if self.bias is None else self.bias.double()
        if self.gating == 2:
            s = torch.sigmoid(logit)
            return s + b, s, err / 4 + 10 * H * (s + abs(b) if self.bias is not None else s), err
        logit = logit + b
        err = err + H * logit.abs()
        return logit, (torch.softmax(logit, -1) if self.gating == 0 else torch.sigmoid(logit)), err, err

    def check_routing(self, x, idx, gate):
        key, score, err, logit_err = self.keys(x)
        idx = idx.long()
        for t in range(x.shape[0]):
            assert len(set(idx[t].tolist())) == self.k
        picked, picked_err = key.gather(1, idx), err.gather(1, idx)
        # in order, and no expert left out that is better than one picked, beyond the bounds
        assert bool((picked[:, 1:] <= picked[:, :-1] + picked_err[:, 1:] + picked_err[:, :-1]).all())
        rest = (key - err).scatter(1, idx, -torch.inf).amax(1)
        assert bool((rest <= picked[:, -1] + picked_err[:, -1]).all())
        want = score.gather(1, idx)
        if self.gating:
            want = want / want.sum(1, keepdim=True)
        # a relative error of e^(2 err) from the logits, then expf (2 ulp), sums of up to 64 terms and a division
        bound = want * (torch.expm1(2 * logit_err.amax(1, keepdim=True)) + 90 * H) + 2.0 ** -126
        assert bool(((gate.double() - want).abs() <= bound).all())

    def ffn(self, e, x):
        """FFN_e(x) of rows x and its bound."""
        (gq, gs), (uq, us), (dq, ds) = self.ffn_of(e)
        a = U.values_rows(*U.quantize_rows(x.float()))
        wg, wu, wd = U.values_weight(gq, gs), U.values_weight(uq, us), U.values_weight(dq, ds)
        g, u = a @ wg.t(), a @ wu.t()
        bg, bu = U.product_bound(a, wg, self.d), U.product_bound(a, wu, self.d)
        act = torch.sigmoid(g) * g
        v = act * u
        # |silu'| < 1.1; expf is off by 2 ulp, then an addition, a division and a product
        bv = 1.1 * bg * (u.abs() + bu) + act.abs() * bu + 9 * H * v.abs() + 2.0 ** -100
        m, h = v.shape
        q, s = U.quantize_rows(v.float())
        hid, off = torch.zeros(m, h, dtype=F64), torch.zeros(m, h, dtype=F64)
        for b in range(U.blocks(h)):
            at = (slice(None), slice(b * BLOCK, (b + 1) * BLOCK))
            sc = s[:, b:b + 1].double()
            bs = bv[at].amax(1, keepdim=True) / U.TOP + 2 * H * sc
            low = sc - bs
            ratio = torch.where(sc > 0, v[at] / sc, 0.0)  # a block of zeros has zero codes
            br = torch.where(low > 0, (bv[at] + ratio.abs() * bs) / low + 2 * H * ratio.abs(), torch.inf).nan_to_num(1e9, 1e9)
            lo, hi = U.e4m3(ratio - br), U.e4m3(ratio + br)
            code = q[at]
            hid[at] = code * sc
            off[at] = code.abs() * bs + torch.maximum(hi - code, code - lo).clamp(min=0) * (sc + bs)
        return hid @ wd.t(), off @ wd.abs().t() + U.product_bound(hid.abs() + off, wd, h)

    def check(self, x, y, idx, gate, counts=None):
        T = x.shape[0]
        self.check_routing(x, idx, gate)
        gate = gate.double()
        ref, bound = self.ffn(self.E, x)
        size = ref.abs() + bound
        for e in idx.unique().tolist():
            t, j = (idx == e).nonzero(as_tuple=True)
            f, b = self.ffn(e, x[t])
            w = gate[t, j, None]
            ref[t] += w * f
            bound[t] += w * b
            size[t] += w * (f.abs() + b)
        # k fused additions
        U.assert_within(y, ref, bound + self.k * H * size, y.dtype)
        if counts is not None:
            want = torch.bincount(idx.flatten().long(), minlength=self.E).int()
            assert torch.equal(counts[:-1], want) and int(counts[-1]) == T


def outputs(c, T):
    return (torch.full((T, c.k), -1, dtype=torch.int32, device="cuda"), torch.full((T, c.k), -1.0, device="cuda"),
            torch.full((c.E + 1,), -1, dtype=torch.int32, device="cuda"))


def forward(layer, c, x, **kw):
    idx, gate, counts = outputs(c, x.shape[0])
    y = layer.forward(x.cuda(), topk_idx=idx, topk_gate=gate, expert_counts=counts, **kw)
    return y, idx.cpu(), gate.cpu(), counts.cpu()


# tokens, d, h, hs, experts, k, gating, bias: the smallest sizes; blocks of 128 that end early in d, h and hs; more
# ranks than hidden or output rows; one expert for every token (several clusters of 16); a shared expert much wider
CASES = [(1, 64, 32, 32, 1, 1, 0, False), (2, 96, 32, 96, 4, 2, 1, True), (5, 256, 128, 128, 60, 4, 0, True),
         (8, 128, 384, 1536, 60, 4, 2, True), (9, 1056, 288, 160, 33, 8, 1, False), (16, 544, 224, 32, 2, 2, 2, False),
         (17, 64, 160, 64, 1, 1, 0, False), (31, 320, 96, 416, 7, 3, 0, False), (33, 192, 64, 32, 3, 1, 2, True),
         (64, 256, 128, 160, 8, 8, 0, False), (64, 1024, 64, 64, 64, 6, 0, True), (3, 2048, 1024, 512, 5, 2, 0, False)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_layer(fp8, case, dtype):
    T, *rest = case
    c = Case(*rest, seed=sum(case))
    x = c.x(T)
    c.check(x, *forward(c.layer(fp8), c, x, out_dtype=dtype))


def test_tokens_do_not_depend_on_their_batch(fp8):
    """A token's output is the same bits alone and in any batch; a repeated call gives the same bits."""
    c = Case(320, 160, 224, 20, 4, seed=3)
    layer, x = c.layer(fp8), c.x(40).cuda()
    whole = layer.forward(x)
    assert torch.equal(whole, layer.forward(x))
    for a, b in ((0, 1), (7, 15), (16, 33), (39, 40)):
        assert torch.equal(layer.forward(x[a:b]), whole[a:b])


def test_ties_go_to_the_lowest_index(fp8):
    c = Case(256, 64, 64, 60, 4, seed=4)
    c.router[:] = c.router[:, :1]
    x = c.x(10)
    _, idx, gate, _ = forward(c.layer(fp8), c, x)
    assert torch.equal(idx, torch.arange(4, dtype=torch.int32).expand(10, 4))
    assert bool((gate.double() - 1 / 60).abs().max() < 1e-8)


@pytest.mark.parametrize("gating", [0, 1, 2])
def test_not_finite_rows_stay_apart(fp8, gating):
    c = Case(192, 96, 64, 6, 2, gating=gating, seed=5)
    layer, x = c.layer(fp8), c.x(20)
    clean = forward(layer, c, x)[0]
    bad = x.clone()
    bad[0, 3], bad[7, 150], bad[19, 0] = float("nan"), float("inf"), float("-inf")
    y, idx, _, counts = forward(layer, c, bad)
    rows = [0, 7, 19]
    assert torch.isnan(y[rows]).all()
    keep = [i for i in range(20) if i not in rows]
    assert torch.equal(y[keep], clean[keep])
    assert bool((idx >= 0).all()) and bool((idx < 6).all()) and int(counts[:-1].sum()) == 40


def test_zero_rows_and_zero_weights(fp8):
    c = Case(256, 128, 128, 8, 2, seed=6)
    c.kinds[0] = tuple((torch.zeros_like(q), torch.zeros_like(s)) for q, s in c.kinds[0])
    x = c.x(6)
    x[2] = 0
    y, idx, gate, counts = forward(c.layer(fp8), c, x)
    c.check(x, y, idx, gate, counts)
    assert bool((y[2] == 0).all())


def test_nothing_outside_the_outputs(fp8):
    c = Case(96, 64, 32, 5, 2, seed=7)
    layer, x = c.layer(fp8), c.x(11).cuda()
    want = layer.forward(x)
    buf = torch.full((15, 96), -3.0, device="cuda")
    y = buf[2:13]
    assert layer.forward(x, y) is y
    assert torch.equal(y, want)
    y.fill_(-3.0)
    assert bool((buf == -3.0).all())
    assert layer.forward(x[:0]).shape == (0, 96)


def test_captured_streams_and_workspaces(fp8):
    """Two captured graphs replayed at once on two streams, and eager calls on a third, do not disturb one another."""
    c = Case(512, 256, 256, 24, 4, seed=8)
    layer = c.layer(fp8)
    xs = [c.x(T, seed=T).cuda() for T in (8, 64, 3)]
    want = [layer.forward(x, out_dtype=BF16) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    graphs, held = [], []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(layer.forward(x, out_dtype=BF16))
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = layer.forward(xs[2], out_dtype=BF16, stream=streams[2])
    torch.cuda.synchronize()
    for a, b in zip([*held, eager], want):
        assert torch.equal(a, b)
    fresh = c.x(8, seed=123).cuda()
    xs[0].copy_(fresh)
    graphs[0].replay()
    assert torch.equal(held[0], layer.forward(fresh, out_dtype=BF16))


def test_refusals(fp8):
    c = Case(64, 32, 32, 4, 2, seed=9)
    layer = c.layer(fp8, max_tokens=16)
    x = c.x(8).cuda()
    for bad, word in ((x.float(), "bfloat16"), (x[:, :32], "d_model"), (x.t().contiguous().t(), "contiguous"),
                      (x.cpu(), "CUDA")):
        with pytest.raises(ValueError, match=word):
            layer.forward(bad)
    with pytest.raises(_error(), match="T=17"):
        layer.forward(c.x(17).cuda())
    with pytest.raises(ValueError, match="y must be"):
        layer.forward(x, torch.empty(8, 32, device="cuda"))
    with pytest.raises(ValueError, match="topk_idx"):
        layer.forward(x, topk_idx=torch.empty(8, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="load"):
        fp8.FP8MoELayer(64, 32, n_experts=4, top_k=2).forward(x)
    with pytest.raises(ValueError, match="w_down"):
        layer.load(*[t if i != 4 else t[:, :, :16] for i, t in enumerate(layer._keep)])


def _error():
    from moe_ffn_layer_fp32_b200 import _lib
    return _lib.MMoEError
