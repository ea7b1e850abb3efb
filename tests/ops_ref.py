"""Plain 64-bit implementations of the operators around the layer, and the error bounds the GPU
tests hold them to (imported by tests, not collected). CPU tensors and numpy arrays throughout."""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24          # half a step of fp32, relative


# ------------------------------------------------------------------ residual add + RMS norm

def norm_ref(x, residual, weight, eps, offset):
    """(h in the rows' type, v in float64)."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hd = h.double()
    r = 1 / torch.sqrt(hd.square().mean(1, keepdim=True) + eps)
    return h, hd * r * (weight.double() + offset)


def norm_rel(H):
    """Relative error of the fp32 v: the sum of squares over at most 64 values a thread and 10 further
    additions errs by (74 + 1) u, of which the square root passes on half; the mean, the root, the
    reciprocal, the weight's offset and the two products add one u each."""
    return (0.5 * min(H, 75) + 8) * U32


def half_step(t, ref):
    """Half a step of type t at |ref| (absolute, with the subnormal step as the least)."""
    tiny = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[t]
    return ref.abs() * (torch.finfo(t).eps / 2) + tiny


# ------------------------------------------------------------------ gated routing

def gate_ref(logits, top_k, score, n_groups=1, topk_groups=1, group_score="max", renorm=True, scale=1.0,
             bias=None):
    """(idx [T, k], w [T, k] float64) by plain loops over sorted lists."""
    T, E = logits.shape
    idx = np.empty((T, top_k), np.int64)
    w = np.zeros((T, top_k), np.float64)
    size = E // n_groups
    for t in range(T):
        l = logits[t].astype(np.float64)
        masked = np.isnan(l) | (l == -np.inf)
        s = np.zeros(E)
        on = ~masked
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[on] = 1 / (1 + np.exp(-l[on]))
        elif on.any():
            top = l[on].max()
            with np.errstate(invalid="ignore"):
                p = np.where(l[on] == top, 1.0, np.exp(l[on] - top))
            s[on] = p / p.sum()
        key = s if bias is None else s + bias.astype(np.float64)
        masked |= np.isnan(key) | (key == -np.inf)
        key = np.where(masked, -np.inf, key)
        allowed = list(range(n_groups))
        if n_groups > 1:
            def rank(g):
                best = sorted((float(key[e]) for e in range(g * size, (g + 1) * size) if not masked[e]), reverse=True)
                if not best:
                    return -math.inf
                return best[0] + best[1] if group_score == "top2" and len(best) > 1 else best[0]
            allowed = sorted(range(n_groups), key=lambda g: (-rank(g), g))[:topk_groups]
        cand = [e for g in allowed for e in range(g * size, (g + 1) * size)]
        chosen = sorted(cand, key=lambda e: (-key[e], e))[:top_k]
        ws = np.array([0.0 if masked[e] else s[e] for e in chosen])
        if renorm:
            ws = ws / ws.sum() if ws.sum() > 0 else np.zeros(top_k)
        idx[t], w[t] = chosen, ws * scale
    return idx, w


def block_map_ref(idx, E, bm):
    hist = np.bincount(idx.reshape(-1), minlength=E)
    off = np.concatenate([[0], np.cumsum(hist)])
    return np.array([[e, off[e] + i, min(bm, hist[e] - i)] for e in range(E) for i in range(0, hist[e], bm)],
                    np.int64).reshape(-1, 3)


# ------------------------------------------------------------------ int4 projection with adapters

def dequant(q, s, b):
    g = [torch.repeat_interleave(t.double(), 64, dim=1) for t in (s, b)]
    return q.double() * g[0] + g[1]


def project_ref(x, q, s, b, A=None, Bm=None, ranks=None, scales=None, of=None, wide=False):
    """(y float64, bound on the error of the rounded result).

    fp32 sums: a sum of n products taken in any order errs by at most (n + 1) u times the sum of the
    products' magnitudes. W's part is held as x . (128 + q) s + (b - 128 s) sum(x) per group (exact
    codes) or as x . bf16(w) (wide: another half step of bf16 a weight)."""
    K = x.shape[1]
    w = dequant(q, s, b)
    xd = x.double()
    y = xd @ w.t()
    bf = torch.finfo(torch.bfloat16).eps / 2
    if wide:
        err = xd.abs() @ w.abs().t() * (bf + (K + 2) * U32)
    else:
        g = [torch.repeat_interleave(t.double(), 64, dim=1) for t in (s, b)]
        size = (128 + q.double()) * g[0].abs() + (g[1] - 128 * g[0]).abs()
        err = xd.abs() @ size.t() * ((64 + 2 * (K // 64) + 4) * U32)
    if A is not None:
        n, R = A.shape[:2]
        for a in range(n):
            at = (of == a).nonzero()[:, 0]
            r = R if ranks is None else int(min(max(int(ranks[a]), 0), R))
            if not len(at) or r == 0:
                continue
            sc = 1.0 if scales is None else float(scales[a])
            Aa, Ba = A[a, :r].double(), Bm[a, :, :r].double()
            z = xd[at] @ Aa.t() * sc
            y[at] += z @ Ba.t()
            # z: K products in fp32, the scale, and a split into two bf16 halves (16 bits)
            dz = xd[at].abs() @ Aa.abs().t() * abs(sc) * ((K + 2) * U32) + z.abs() * 2.0 ** -16
            err[at] += (dz + z.abs() * ((2 * r + 4) * U32)) @ Ba.abs().t()
    err = err + (y.abs() + err) * bf + 2.0 ** -134
    return y, err
