"""Plain 64-bit implementations of the attention-side operators and the error
bounds of the HIP kernels against them, for the tests (CPU only).

Bounds.  A rounding to a type is off by at most half a step, eps / 2 of the
value.  Of a softmax-weighted mean out = sum p v / sum p the kernels round each
weight to 16 bits (at most u_p of it, or 2^-25 of the largest weight where the
fp16 weight is subnormal), make each score with fp32 sums of D products (at
most (D + 8) 2^-24 sum |q k|), take exp2 of an argument x in fp32 (2^-23 (2 +
|x|)), add up to N weights (N 2^-24) and round once at the end."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def norm_rope(x, w, cos, sin, pos, eps, inter):
    """x [T][H][D]; (result, |a| + |b| of every value) in float64; tokens with a
    position outside the table give NaN."""
    x = x.double()
    T, H, D = x.shape
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    half = cos.shape[1]
    ok = (pos >= 0) & (pos < cos.shape[0])
    c = cos.double()[pos.long().clamp(0, cos.shape[0] - 1)][:, None, :]
    s = sin.double()[pos.long().clamp(0, cos.shape[0] - 1)][:, None, :]
    ia = torch.arange(0, 2 * half, 2) if inter else torch.arange(half)
    ib = ia + 1 if inter else ia + half
    out, mag = n.clone(), n.abs()
    a, b = n[..., ia], n[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    out[~ok] = float("nan")
    return out, mag


def norm_rope_bound(want, mag, dtype):
    # mean of squares, reciprocal root, three products and the rotation: 32
    # roundings of 2^-24 at most
    return HALF[dtype] * want.abs() + 32 * 2.0 ** -24 * mag + TINY[dtype]


def attend(q, k, v, seen, scale, v_scale_max, dtype, weight_half):
    """q [m][D], k and v [n][D] float64, seen [m][n] bool.  Returns (out, bound,
    lse, lse bound); a row that sees nothing gives zeros and -inf."""
    m, D = q.shape
    n = k.shape[0]
    out = torch.zeros((m, D), dtype=torch.float64)
    bound = torch.zeros((m, D), dtype=torch.float64)
    lse = torch.full((m,), -math.inf, dtype=torch.float64)
    lse_b = torch.zeros((m,), dtype=torch.float64)
    live = seen.any(-1)
    if n == 0 or not bool(live.any()):
        return out, bound, lse, lse_b
    qs, se = q[live], seen[live]
    s = qs @ k.T * scale
    big = qs.abs() @ k.abs().T * scale
    s = s.masked_fill(~se, -math.inf)
    mx = s.amax(-1, keepdim=True)
    p = torch.exp(s - mx)
    l = p.sum(-1, keepdim=True)
    o = p @ v / l
    arg = torch.where(se, (s - mx).abs(), torch.zeros_like(s)) * 1.4427 + mx.abs() * 1.4427
    # weights below 2^-30 of the largest add nothing that counts, whatever their own error
    delta = torch.where(p > 2.0 ** -30, (D + 8) * 2.0 ** -24 * big + 2.0 ** -23 * (2 + 2 * arg), torch.zeros_like(p))
    rel = (p * delta).sum(-1, keepdim=True) / l + n * 2.0 ** -24
    mean_abs = p @ v.abs() / l
    # 2^-25 of the largest weight times its scale (within a factor of two of the largest scale), integers up to 15
    small = n * 2.0 ** -25 * 2 * v_scale_max / l if weight_half == 2.0 ** -11 else 0.0
    b = HALF[dtype] * o.abs() + TINY[dtype] + weight_half * mean_abs + (p * delta) @ v.abs() / l + rel * o.abs() + small
    out[live], bound[live] = o, b * 1.01
    lse[live] = (mx + torch.log(l))[:, 0]
    lse_b[live] = (rel[:, 0] + delta.amax(-1) + 2.0 ** -22 * (2 + lse[live].abs()))
    return out, bound, lse, lse_b


def check(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got {float(got[i])}, "
                             f"want {float(want[i])} +- {float(bound[i])}")


def values(seed, shape, dtype, scale=1.0, wide=0.02):
    """Normal values, a few channels eight times larger, in a 16-bit type (CPU)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32) * scale
    x *= np.where(rng.random(shape[1:]) < wide, 8.0, 1.0).astype(np.float32)
    return torch.from_numpy(x).to(dtype)
