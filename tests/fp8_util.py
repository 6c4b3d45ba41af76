"""Plain 64-bit forms of the e4m3 operators, written apart from the library, and their error bounds."""
from __future__ import annotations

import torch

BLOCK, TOP = 128, 448.0


def blocks(n):
    return -(-n // BLOCK)


def e4m3(v):
    """Nearest e4m3 value (ties to even, saturating) of 64-bit v; NaN stays NaN."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -40)).exponent.double() - 1
    step = torch.exp2(e.clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def scale_of(amax):
    """max|v| / 448 in FP32: a 64-bit quotient of FP32 numbers rounded once is the FP32 quotient."""
    return (amax.double() / TOP).float()


def code_of(v, s):
    """The values that the codes of FP32 v stand for under scales s (both broadcast), 0 where s is not positive."""
    s = s.double().expand_as(v)
    return e4m3(torch.where(s > 0, (v.double() / s).float().double(), torch.zeros_like(v, dtype=torch.float64)))


def quantize_rows(v):
    """FP32 [M, K] -> code values (float64) and scales (float32)."""
    m, k = v.shape
    q = torch.zeros(m, k, dtype=torch.float64)
    s = torch.zeros(m, blocks(k), dtype=torch.float32)
    for b in range(blocks(k)):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = scale_of(part.abs().amax(1))
        q[:, b * BLOCK:(b + 1) * BLOCK] = code_of(part, s[:, b:b + 1])
    return q, s


def quantize_blocks(w):
    n, k = w.shape
    q = torch.zeros(n, k, dtype=torch.float64)
    s = torch.zeros(blocks(n), blocks(k), dtype=torch.float32)
    for i in range(blocks(n)):
        for j in range(blocks(k)):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            s[i, j] = scale_of(w[at].abs().amax())
            q[at] = code_of(w[at], s[i, j])
    return q, s


def values_rows(q, s):
    return q.double() * s.double().repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def values_weight(q, s):
    n, k = q.shape
    return q.double() * s.double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def product_bound(a, w, k):
    """Largest error of an FP32 product of values a [M, K] and w [N, K], element by element.

    Each block adds 128 products of codes, exact in FP32, at most one rounding of a step (2^-23) each on the tensor
    cores; then come the product of the two scales, the scaled addition and one addition a block (2^-24 each).  The product of two scales may be subnormal: it is then off by
    at most half of the smallest subnormal (2^-150), which a block's sum of 128 products of codes (448^2 at most each)
    multiplies, and so may be the block's scaled sum."""
    tiny = blocks(k) * (128 * 448 ** 2 + 1) * 2.0 ** -150
    return tiny + ((128 * 2 + blocks(k) + 8 + 2) * 2.0 ** -24) * (a.abs() @ w.abs().t())


def assert_within(got, ref, bound, dtype):
    """|got - ref| <= bound, plus half a step of BF16 where that is what got was rounded to."""
    got = got.detach().double().cpu()
    if dtype == torch.bfloat16:
        bound = bound + (ref.abs() + bound) * 2.0 ** -8
    over = (got - ref).abs() - bound
    assert got.shape == ref.shape
    assert bool((over <= 0).all()), f"{int((over > 0).sum())} of {over.numel()} outside, worst by {over.max().item():.3g}"
