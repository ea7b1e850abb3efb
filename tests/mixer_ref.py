"""Plain 64-bit implementations of the operators of a block's mixer half, and the error bounds the GPU tests
hold them to (imported by tests, not collected). CPU tensors throughout."""
from __future__ import annotations

import math

import torch

from ops_ref import U32, half_step, norm_rel

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


# ------------------------------------------------------------------ int8 projection

def int8_ref(w, w_scales, x, x_scales, bias):
    """(y in float64, its bound before the output's rounding): the whole number to fp32, two products and the bias round
    once each."""
    y = (x.double() @ w.double().t()) * x_scales.double()[:, None] * w_scales.double()
    err = 3 * U32 * y.abs() * (1 + 4 * U32)
    if bias is not None:
        y = y + bias.double()
        err = err + U32 * (y.abs() + err)
    return y, err


# ------------------------------------------------------------------ rotary positions

def rope_ref(x, positions, radians, rot, interleaved, magnitude=1.0, inverse=False):
    """(turned [T, heads, D] in float64, its bound before the output's rounding).

    Cosine and sine err by at most 4 u: the angle's rest (at most an eighth of a turn) is rounded to fp32 and multiplied
    by 2 pi 2^-32 (2 u of at most 0.79), the series' last steps round twice, and its cut and the 2^-32 turns that are left
    out stay below 5e-9 (u / 10). The magnitude is the fifth, the products and the sum two more."""
    angle = positions.double()[:, None] * radians.double()
    cos, sin = (f(angle)[:, None] * magnitude for f in (torch.cos, torch.sin))
    if inverse:
        sin = -sin
    y, err = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    half = rot // 2
    ia, ib = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * cos - b * sin, a * sin + b * cos
    # (float64's own angle is off by 2^-53 of it)
    e = (7.5 * U32 + angle.abs()[:, None] * 2.0 ** -52) * abs(magnitude) * (a.abs() + b.abs())
    err[..., ia], err[..., ib] = e, e
    return y, err


# ------------------------------------------------------------------ linear attention

def linear_ref(q, k, v, g, starts, cu, scale):
    """Token after token in float64: (o, bound on o before its rounding where nothing is rounded to bf16, the sum that a
    bf16 operand's rounding scales with, states, S_abs). g [T, Hv]; starts [n, Hv, dk, dv]."""
    T, Hv, dv = v.shape
    dk, each = q.shape[2], Hv // q.shape[1]
    o, weight = torch.zeros((T, Hv, dv), dtype=torch.float64), torch.zeros((T, Hv, dv), dtype=torch.float64)
    q, k = (t.double().repeat_interleave(each, 1) for t in (q, k))
    v, g = v.double(), g.double()
    states, sums = starts.double().clone(), starts.double().abs()
    for i in range(len(cu) - 1):
        S, A = states[i].clone(), sums[i].clone()
        for t in range(int(cu[i]), int(cu[i + 1])):
            d = torch.exp(g[t])[:, None, None]
            S = torch.where(d == 0, 0.0, S * d) + k[t][:, :, None] * v[t][:, None, :]
            A = torch.where(d == 0, 0.0, A * d) + (k[t][:, :, None] * v[t][:, None, :]).abs()
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
            weight[t] = abs(scale) * (q[t][:, :, None].abs() * A).sum(1)
        states[i], sums[i] = S, A
    return o, weight, states, sums


def linear_bound(dk, length, chunked):
    """(relative to the absolute sums of o: the state's and products' fp32 roundings and bf16 operands; of the state).

    A term of the state passes, per chunk of 64 tokens (per token for the walk), one product by a decay (of 2 u: the
    exponential's own ulp and its argument's, whose size e^-x x limits to 0.4 u more in all) and a sum of up to 64 terms; o
    adds a sum over dk and, for a chunk, over 64 tokens. With bf16 operands each product of o carries one more 2^-8."""
    steps = (length + 63) // 64 * 70 + 10 if chunked else 4 * length + 10
    state = steps * U32
    return state + (dk + 70) * U32 + (1.01 * BF16_HALF if chunked else 0.0), state


# ------------------------------------------------------------------ the norm after a block

def gated_ref(x, c, weight=None, gate=None, channel=None, residual=None, next_weight=None):
    """(v before the second norm, its bound, v after it or None, its bound) in float64."""
    T, H = x.shape
    u, rel = x.double(), 0.0
    if c["normalize"]:
        G = c["group"] or H
        f = u.view(T, -1, G)
        w = 1.0 if weight is None else (weight.double() + c["offset"]).repeat(H // G)
        u = (f / torch.sqrt(f.square().mean(2, keepdim=True) + c["eps"])).reshape(T, H) * w
        rel = norm_rel(G) + 3 * U32
    if gate is not None:
        z = gate.double()
        u = u * torch.sigmoid(z) * (z if c["gate"] == 1 else 1.0)
        # the exponential (its part put back, its ulp, their product), 1 + e, the reciprocal's ulp, z and the product; for
        # rows of 16 bits nothing is put back: log2(e) and its product with z round, 2 u |z| log2(e) of the exponent in base
        # 2, of which ln 2 reach the result
        rel = rel + 10 * U32 + (2 * U32 * z.abs() if x.dtype != torch.float32 else 0.0)
    u = u * c["scale"] * (1.0 if channel is None else channel.double())
    rel += 4 * U32
    err = rel * u.abs() + 2.0 ** -126
    v = u
    if residual is not None:
        v = u + residual.double()
        err = err + U32 * (v.abs() + err)
    if next_weight is None:
        return v, err, None, None
    r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + c["eps"])
    y = v * r * (next_weight.double() + c["offset"])
    # the root's relative error from v's: at most the ratio of the two's root mean squares
    off = err.square().mean(1, keepdim=True).sqrt() * r + norm_rel(H) + 2 * U32
    return v, err, y, off * y.abs() * (1 + off) + err * r * (next_weight.double() + c["offset"]).abs() * (1 + off)
