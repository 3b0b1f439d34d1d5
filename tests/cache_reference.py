"""The paged cache's operators from their definition, in float64 on the CPU, and how far the kernels
may be from it.

Stored e4m3 rows: value = code * 2^e with the smallest e for which max|x| <= 448 * 2^e, |e| <= 50, code = x * 2^-e rounded to nearest even to three fraction bits (steps of 2^-9 below 2^-6).
"""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.bfloat16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -8}     # of the output's type


def quantise(x):
    """(values that the codes stand for, exponents) of rows, in float64."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, -50.0)
    while bool((more := (top > 448.0 * torch.exp2(e)) & (e < 50)).any()):
        e = torch.where(more, e + 1, e)
    y = (x / torch.exp2(e)).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e), e[..., 0]


def attention(q, k, v, pos, causal, window, scale):
    """One head: q [m, d] at positions pos, k and v [n, d], all float64.  Returns the output [m, d], the
    log of the softmax sum [m], and what the bounds need: the weighted mean of |v|, the largest |q||k|
    sum of a visible logit, and how many keys each row sees.  Keys that a row does not see are left out
    of its sums altogether."""
    m, d = q.shape
    n = k.shape[0]
    o, lse = torch.zeros(m, v.shape[1], dtype=torch.float64), torch.full((m,), -math.inf, dtype=torch.float64)
    mean_abs, size, seen = torch.zeros_like(o), torch.zeros(m, dtype=torch.float64), torch.zeros(m, dtype=torch.float64)
    j = torch.arange(n)
    for r in range(m):
        keep = torch.ones(n, dtype=torch.bool)
        if causal:
            keep &= j <= pos[r]
        if window:
            keep &= j > pos[r] - window
        if not bool(keep.any()):
            continue
        kk, vv = k[keep], v[keep]
        s = scale * (kk @ q[r])
        lse[r] = torch.logsumexp(s, 0)
        w = torch.exp(s - lse[r])
        o[r], mean_abs[r] = w @ vv, w @ vv.abs()
        size[r] = scale * (kk.abs() @ q[r].abs()).max()
        seen[r] = kk.shape[0]
    return dict(o=o, lse=lse, mean_abs=mean_abs, size=size, seen=seen, vmax=v.abs().max() if n else 0.0)


def bounds(ref, dtype, d):
    """(bound of |o - ref.o|, bound of |lse - ref.lse|), element by element.

    * A logit is a sum of d products in fp32; each of its d additions (the tensor core may cut instead of
      round) loses at most 2^-23 of the sum of magnitudes, its scaling and the subtraction of the
      maximum 2^-23 of its size each: E = (d + 4) 2^-23 size, absolutely, and that is the relative error of
      its weight, plus 2^-21 for the exponential.
    * Weights enter the product with v in the type of the values (bf16, off by 2^-8 relative at most) or in
      fp16 for e4m3 pools (2^-11, or 2^-25 of the largest weighted row where they fall below fp16's normal
      range: at most n * 2^-24 max|v| in all) or in fp32.
    * Sums over the n visible keys lose at most n 2^-23 relative to the sum of magnitudes, above and below
      the division: 2 n 2^-23 mean|v|.
    * The output is rounded once.
    """
    weight = {"bf16": 2.0 ** -8, "fp32": 0.0, "e4m3": 2.0 ** -11}[dtype]
    logit = (d + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -21
    n = ref["seen"]
    rel = weight + 2 * logit + 2 * n * 2.0 ** -23
    o = ref["mean_abs"] * rel[:, None] * 1.01 + HALF_STEP[dtype] * ref["o"].abs() + 1e-37
    if dtype == "e4m3":
        o = o + (n * 2.0 ** -24)[:, None] * ref["vmax"]
    return o, logit + n * 2.0 ** -23 + 2.0 ** -22 * (1 + ref["lse"].abs().nan_to_num(0, 0, 0))
