"""Cases and plain forms of the 8-bit floating-point operators and of the block norm.

Four operators, all next to the MoE feed-forward layer of this package:

  linear   a matrix product in 8-bit floating point (e4m3): activations quantised per token and 128
           input features, weights per block of 128 x 128
  experts  the same product over rows sorted by expert, each group with its own weights
  moe      the whole MoE layer (router, top-k, SwiGLU experts, shared expert, combine) on such weights
           for up to 64 tokens
  norm     the norms after and before a block, fused with the block's gate and the residual update

`own` false: plain torch in 32 bits (router logits in 64); true: the package's operators.

Definitions.  A quantised block has s = max|v| / 448 (an IEEE FP32 division; 0 for a block of zeros)
and the codes e4m3(v / s) (IEEE FP32 division, round to nearest even; 0 where s is 0).
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # largest finite e4m3 value
EPS = 1e-6   # of the norms

# ---------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one decode token through a projection: nothing but latency and one pass over the weights
        {"name": "linear 1 token", "op": "linear", "tokens": 1, "n": 2048, "k": 1024, "out": "bf16"},
        # a decode batch: still bound by the weights
        {"name": "linear 64 tokens", "op": "linear", "tokens": 64, "n": 4096, "k": 2048, "out": "bf16"},
        # the ragged end of a prompt, sizes that end inside every tile and block, FP32 output
        {"name": "linear ragged", "op": "linear", "tokens": 777, "n": 1000, "k": 784, "out": "f32"},
        # four prompts of 8192 tokens: bound by the tensor cores
        {"name": "linear prefill", "op": "linear", "tokens": 32768, "n": 2048, "k": 2048, "out": "bf16"},
        # gate and up projections of 60 experts for a prompt of 2048 tokens, four experts each
        {"name": "experts 2048 tokens", "op": "experts", "rows": 8192, "groups": 60, "n": 1024, "k": 1024,
         "skew": 0.0, "out": "bf16"},
        # the same for 8192 tokens with a load skewed by about ten to one
        {"name": "experts skewed", "op": "experts", "rows": 32768, "groups": 60, "n": 1536, "k": 1536,
         "skew": 0.25, "out": "bf16"},
        # one decode token: five experts' weights
        {"name": "moe 1 token", "op": "moe", "tokens": 1, "d": 1024, "h": 512, "hs": 512, "experts": 60, "top": 4,
         "gating": 0, "bias": False},
        # eight sequences on the layer shape with a wide shared expert, sigmoid gates, selection bias
        {"name": "moe 8 tokens", "op": "moe", "tokens": 8, "d": 768, "h": 384, "hs": 1536, "experts": 60, "top": 4,
         "gating": 2, "bias": True},
        # the largest decode batch: every expert's weights
        {"name": "moe 64 tokens", "op": "moe", "tokens": 64, "d": 2048, "h": 1024, "hs": 1024, "experts": 60,
         "top": 4, "gating": 0, "bias": False},
        # between two blocks of a decode step, with the codes that the next product reads
        {"name": "norm 1 token", "op": "norm", "tokens": 1, "d": 1024, "res": "bf16", "y": "f32", "gate": "channel",
         "post": True, "codes": True},
        # a ragged prompt with an FP32 residual stream and a gate for each token
        {"name": "norm ragged", "op": "norm", "tokens": 2049, "d": 768, "res": "f32", "y": "f32", "gate": "token",
         "post": True, "codes": False},
        # four prompts of 8192 tokens: bound by memory
        {"name": "norm prefill", "op": "norm", "tokens": 32768, "d": 2048, "res": "bf16", "y": "f32",
         "gate": "channel", "post": True, "codes": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "experts", "moe", "norm"])
    if op == "linear":
        n, k = _log(rng, 64, 4096), 16 * _log(rng, 8, 128)
        most = min(32768, 32768 * 2048 * 2048 // (n * k))
        return {"op": op, "tokens": _log(rng, 1, most), "n": n, "k": k, "out": rng.choice(["bf16", "f32"])}
    if op == "experts":
        n, k = 8 * _log(rng, 16, 192), 16 * _log(rng, 8, 96)
        return {"op": op, "rows": _log(rng, 4, 32768), "groups": rng.randint(2, 64), "n": n, "k": k,
                "skew": rng.choice([0.0, 0.25, 0.5]), "out": rng.choice(["bf16", "f32"])}
    if op == "moe":
        gating = rng.choice([0, 1, 2])
        return {"op": op, "tokens": _log(rng, 1, 64), "d": 32 * _log(rng, 8, 64), "h": 32 * _log(rng, 4, 32),
                "hs": 32 * _log(rng, 4, 32), "experts": rng.randint(8, 60), "top": rng.randint(1, 8),
                "gating": gating, "bias": rng.random() < 0.5}
    return {"op": op, "tokens": _log(rng, 1, 32768), "d": 8 * _log(rng, 16, 256), "res": rng.choice(["bf16", "f32"]),
            "y": rng.choice(["bf16", "f32"]), "gate": rng.choice(["none", "channel", "token", "full"]),
            "post": rng.random() < 0.7, "codes": rng.random() < 0.5}


# --------------------------------------------------------------------------------------------- inputs

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _blocks(n):
    return -(-n // BLOCK)


def _encode(v, s):
    """e4m3 codes of v for the scales s (same shape or broadcastable), 0 where the scale is."""
    return torch.where(s > 0, v / s, torch.zeros_like(v)).clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _scale(top):
    """max|v| / 448: by a tensor, for torch multiplies by the reciprocal of a Python number."""
    return top / torch.full_like(top, TOP)


def _quantize_rows(v):
    """FP32 [..., K] -> codes and scales of each row's blocks of 128."""
    k = v.shape[-1]
    p = torch.nn.functional.pad(v, (0, _blocks(k) * BLOCK - k)).unflatten(-1, (-1, BLOCK))
    s = _scale(p.abs().amax(-1))
    return _encode(p, s.unsqueeze(-1)).flatten(-2)[..., :k].contiguous(), s


def _quantize_weight(w):
    """FP32 [..., N, K] -> codes and scales of the blocks of 128 x 128."""
    n, k = w.shape[-2:]
    p = torch.nn.functional.pad(w, (0, _blocks(k) * BLOCK - k, 0, _blocks(n) * BLOCK - n))
    p = p.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))  # [..., nb, 128, kb, 128]
    s = _scale(p.abs().amax((-3, -1)))
    q = _encode(p, s.unsqueeze(-2).unsqueeze(-1))
    return q.flatten(-4, -3).flatten(-2)[..., :n, :k].contiguous(), s


def _spread(s, n, dim):
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _decode_rows(q, s):
    return q.float() * _spread(s, q.shape[-1], -1)


def _decode_weight(q, s):
    return q.float() * _spread(_spread(s, q.shape[-1], -1), q.shape[-2], -2)


def _activations(g, rows, k):
    """Activations of a language model: normal, with one feature in 64 much larger."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 1 / 64
    return x * torch.where(big, 12.0, 1.0)


def _expert_weights(g, e, h, d):
    """Gate and up rows (quantised apart, so that no block holds both) and the down projection of e experts."""
    gq, gs = _quantize_weight(0.02 * torch.randn(e, h, d, generator=g, device="cuda"))
    uq, us = _quantize_weight(0.02 * torch.randn(e, h, d, generator=g, device="cuda"))
    dq, ds = _quantize_weight(0.02 * torch.randn(e, d, h, generator=g, device="cuda"))
    return torch.cat([gq.view(torch.uint8), uq.view(torch.uint8)], 1).view(torch.float8_e4m3fn), torch.cat([gs, us], 1), dq, ds


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "linear":
        st["x"] = _activations(g, case["tokens"], case["k"]).bfloat16()
        st["wq"], st["ws"] = _quantize_weight(0.02 * torch.randn(case["n"], case["k"], generator=g, device="cuda"))
    elif op == "experts":
        r, e = case["rows"], case["groups"]
        c = torch.Generator().manual_seed(seed)
        share = (1.0 + torch.randperm(e, generator=c).double()) ** -case["skew"]
        of = torch.multinomial(share, r, replacement=True, generator=c)
        counts = torch.bincount(of, minlength=e)
        st["most"] = int(counts.max())  # rows of the largest group
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int().cuda()
        st["xq"], st["xs"] = _quantize_rows(_activations(g, r, case["k"]).bfloat16().float())
        st["wq"], st["ws"] = _quantize_weight(0.02 * torch.randn(e, case["n"], case["k"], generator=g, device="cuda"))
    elif op == "moe":
        e, d = case["experts"], case["d"]
        st["x"] = torch.randn(case["tokens"], d, generator=g, device="cuda").bfloat16()
        st["router"] = 0.02 * torch.randn(d, e, generator=g, device="cuda")
        st["router_bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        st["gq"], st["gs"], st["dq"], st["ds"] = _expert_weights(g, e, case["h"], d)
        st["sgq"], st["sgs"], st["sdq"], st["sds"] = (t[0] for t in _expert_weights(g, 1, case["hs"], d))
        if own:
            # the object that a program keeps: it holds the tensors above as they are
            from moe_ffn_layer_fp32_b200.fp8 import FP8MoELayer
            layer = FP8MoELayer(d, case["h"], shared_hidden=case["hs"], n_experts=e, top_k=case["top"],
                                gating=case["gating"], has_router_bias=case["bias"])
            layer.load(st["router"], st["router_bias"], st["gq"], st["gs"], st["dq"], st["ds"],
                       st["sgq"], st["sgs"], st["sdq"], st["sds"])
            st["layer"] = layer
    else:
        t, d = case["tokens"], case["d"]
        st["r"] = (3.0 * torch.randn(t, d, generator=g, device="cuda")).to(TYPES[case["res"]])
        st["block"] = torch.randn(t, d, generator=g, device="cuda").to(TYPES[case["y"]])
        shape = {"none": None, "channel": (d,), "token": (t, 1), "full": (t, d)}[case["gate"]]
        st["g"] = None if shape is None else torch.rand(shape, generator=g, device="cuda")
        st["post_w"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["post"] else None
        st["pre_w"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        st["scale"] = 0.875  # what the residual stream is scaled by before the block's output is added
    return st


# ----------------------------------------------------------------------------------------- plain forms


def _linear(st):
    q, s = _quantize_rows(st["x"].float())
    return (_decode_rows(q, s) @ _decode_weight(st["wq"], st["ws"]).t()).to(TYPES[st["out"]])


def _experts(st):
    off, r, e = st["offsets"].long(), st["rows"], st["groups"]
    row = torch.arange(r, device="cuda")
    of = torch.searchsorted(off[1:], row, right=True)
    at = row - off[of]
    x = torch.zeros(e, st["most"], st["k"], device="cuda")
    x[of, at] = _decode_rows(st["xq"], st["xs"])
    return torch.bmm(x, _decode_weight(st["wq"], st["ws"]).transpose(1, 2))[of, at].to(TYPES[st["out"]])


def _route(st):
    """Top-k and gates; the logits in 64 bits, rounded once."""
    logits = (st["x"].double() @ st["router"].double()).float()
    if st["bias"] and st["gating"] != 2:
        logits = logits + st["router_bias"]
    if st["gating"] == 0:
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        key = logits
    else:
        p = 1 / (1 + torch.exp(-logits))
        key = p + st["router_bias"] if st["bias"] and st["gating"] == 2 else (p if st["gating"] == 2 else logits)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : st["top"]]
    gate = p.gather(1, idx)
    return idx, gate if st["gating"] == 0 else gate / gate.sum(-1, keepdim=True)


def _swiglu_codes(gu):
    g, u = gu.chunk(2, -1)
    return _decode_rows(*_quantize_rows(g / (1 + torch.exp(-g)) * u))


def _gate_up(q, s, h):
    return torch.cat([_decode_weight(q[..., :h, :], s[..., : _blocks(h), :]),
                      _decode_weight(q[..., h:, :], s[..., _blocks(h):, :])], -2)


def _moe(st):
    idx, gate = _route(st)
    t, top, h = st["tokens"], st["top"], st["h"]
    x = _decode_rows(*_quantize_rows(st["x"].float()))
    if t * top < st["experts"]:  # few tokens: the chosen experts' weights
        pick = idx.flatten()
        gu = torch.bmm(_gate_up(st["gq"][pick], st["gs"][pick], h), x.repeat_interleave(top, 0).unsqueeze(-1))
        act = _swiglu_codes(gu.squeeze(-1)).unsqueeze(-1)
        each = torch.bmm(_decode_weight(st["dq"][pick], st["ds"][pick]), act).view(t, top, -1)
    else:  # every expert on every token
        gu = torch.matmul(x, _gate_up(st["gq"], st["gs"], h).transpose(1, 2))
        every = torch.bmm(_swiglu_codes(gu), _decode_weight(st["dq"], st["ds"]).transpose(1, 2))
        each = every[idx, torch.arange(t, device="cuda").unsqueeze(1)]
    shared = _swiglu_codes(x @ _gate_up(st["sgq"], st["sgs"], st["hs"]).t()) @ _decode_weight(st["sdq"], st["sds"]).t()
    counts = torch.zeros(st["experts"] + 1, dtype=torch.int32, device="cuda")
    counts[:-1].index_add_(0, idx.flatten(), torch.ones(t * top, dtype=torch.int32, device="cuda"))
    counts[-1] = t
    return ((gate.unsqueeze(-1) * each).sum(1) + shared).bfloat16(), idx.int(), gate, counts


def _norm(st):
    z = st["block"].float()
    if st["post_w"] is not None:
        z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS) * st["post_w"]
    if st["g"] is not None:
        z = st["g"] * z
    r = st["scale"] * st["r"].float() + z
    x = r / torch.sqrt(r.square().mean(-1, keepdim=True) + EPS) * st["pre_w"]
    out = (r.to(st["r"].dtype), x.bfloat16())
    return out + _quantize_rows(x) if st["codes"] else out


def run(state):
    op = state["op"]
    if not own:
        return {"linear": _linear, "experts": _experts, "moe": _moe, "norm": _norm}[op](state)
    if op == "linear":
        from moe_ffn_layer_fp32_b200.fp8 import linear_fp8
        return linear_fp8(state["x"], state["wq"], state["ws"], out_dtype=TYPES[state["out"]])
    if op == "experts":
        from moe_ffn_layer_fp32_b200.fp8 import grouped_gemm_fp8
        return grouped_gemm_fp8(state["xq"], state["xs"], state["offsets"], state["wq"], state["ws"],
                                out_dtype=TYPES[state["out"]])
    if op == "moe":
        t, top, x = state["tokens"], state["top"], state["x"]
        idx = torch.empty((t, top), dtype=torch.int32, device=x.device)
        gate = torch.empty((t, top), dtype=torch.float32, device=x.device)
        counts = torch.empty(state["experts"] + 1, dtype=torch.int32, device=x.device)
        y = state["layer"].forward(x, out_dtype=torch.bfloat16, topk_idx=idx, topk_gate=gate, expert_counts=counts)
        return y, idx, gate, counts
    from moe_ffn_layer_fp32_b200.norm import block_norm
    out = block_norm(state["r"], state["block"], post_weight=state["post_w"], gate=state["g"],
                     residual_scale=state["scale"], pre_weight=state["pre_w"], eps=EPS, quantize=state["codes"])
    return tuple(t for t in out if t is not None)


# ------------------------------------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k = case["tokens"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * m * k + n * k + 4 * _blocks(n) * _blocks(k) + size * m * n, "flops": 2 * m * n * k}
    if op == "experts":
        r, n, k = case["rows"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        busy = case["groups"] * (1 - (1 - 1 / case["groups"]) ** r)  # groups with a row, for an even load
        return {"bytes": r * (k + 4 * _blocks(k)) + busy * (n * k + 4 * _blocks(n) * _blocks(k)) + size * r * n
                + 4 * (case["groups"] + 1), "flops": 2 * r * n * k}
    if op == "moe":
        t, d, h, hs, e, top = (case[n] for n in ("tokens", "d", "h", "hs", "experts", "top"))
        busy = e * (1 - (1 - top / e) ** t)  # experts that some token selects, for an even load
        weights = 3 * d * (busy * h + hs) * (1 + 4 / BLOCK ** 2)
        return {"bytes": weights + 4 * d * e + 4 * t * d + 8 * t * top + 4 * (e + 1),
                "flops": 2 * t * (3 * d * (top * h + hs) + d * e)}
    t, d = case["tokens"], case["d"]
    each = 2 * (2 if case["res"] == "bf16" else 4) + (2 if case["y"] == "bf16" else 4) + 2
    each += (4 if case["gate"] == "full" else 0) + (1 + 4 / BLOCK if case["codes"] else 0)
    return {"bytes": t * d * each + (4 * t if case["gate"] == "token" else 0)
            + 4 * d * (1 + case["post"] + (case["gate"] == "channel")), "flops": 12 * t * d}


# --------------------------------------------------------------------------- the definitions in 64 bits


def _e4m3(v):
    """Nearest e4m3 value (ties to even) of 64-bit v: three fraction bits, no exponent under -6, saturating."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -40)).exponent.double() - 1
    step = torch.exp2(e.clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _stood_for(v):
    """What each row of 64-bit v stands for once quantised in blocks of 128: the FP32 divisions of the definition are
    64-bit divisions of FP32 numbers rounded once to FP32, which is the same."""
    codes, scales = _exact_codes(v)
    return codes * scales.repeat_interleave(BLOCK, -1)[..., : v.shape[-1]]


def _exact_codes(v):
    t, k = v.shape
    codes = torch.zeros(t, k, dtype=torch.float64, device=v.device)
    scales = torch.zeros(t, _blocks(k), dtype=torch.float64, device=v.device)
    for b in range(_blocks(k)):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        s = (part.abs().amax(1) / TOP).float().double()
        ratio = torch.where(s[:, None] > 0, part / s[:, None].clamp(min=1e-300), 0.0)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(ratio.float().double())
        scales[:, b] = s
    return codes, scales


def _weight64(q, s):
    w = q.to(torch.float64)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= s[i, j].double()
    return w


def _ffn64(x, gq, gs, dq, ds, h):
    gate = x @ _weight64(gq[:h], gs[: _blocks(h)]).t()
    up = x @ _weight64(gq[h:], gs[_blocks(h):]).t()
    return _stood_for((gate * torch.sigmoid(gate) * up).float().double()) @ _weight64(dq, ds).t()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _stood_for(st["x"].double()) @ _weight64(st["wq"], st["ws"]).t()
    if op == "experts":
        x = st["xq"].double() * st["xs"].double().repeat_interleave(BLOCK, 1)[:, : case["k"]]
        off = st["offsets"].tolist()
        return torch.cat([x[a:b] @ _weight64(st["wq"][i], st["ws"][i]).t() for i, (a, b) in enumerate(zip(off, off[1:]))])
    if op == "moe":
        logit = st["x"].double() @ st["router"].double()
        b = st["router_bias"].double() if case["bias"] else 0.0
        if case["gating"] == 0:
            score = torch.softmax(logit + b, -1)
            key = logit + b
        elif case["gating"] == 1:
            score = torch.sigmoid(logit + b)
            key = logit + b
        else:
            score = torch.sigmoid(logit)
            key = score + b
        idx = key.topk(case["top"], -1).indices
        gate = score.gather(1, idx)
        if case["gating"] != 0:
            gate = gate / gate.sum(-1, keepdim=True)
        x = _stood_for(st["x"].double())
        y = _ffn64(x, st["sgq"], st["sgs"], st["sdq"], st["sds"], case["hs"])
        for e in idx.unique().tolist():
            t, j = (idx == e).nonzero(as_tuple=True)
            y[t] += gate[t, j, None] * _ffn64(x[t], st["gq"][e], st["gs"][e], st["dq"][e], st["ds"][e], case["h"])
        return y, None, gate, None
    z = st["block"].double()
    if st["post_w"] is not None:
        z = z * (z.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["post_w"].double()
    r = st["scale"] * st["r"].double() + (z if st["g"] is None else st["g"].double() * z)
    x = r * (r.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["pre_w"].double()
    return (r, x) + _exact_codes(x) if case["codes"] else (r, x)
