"""Plain 64-bit definitions of the operators between a layer's products, for the
tests: numpy only, written from the formulas of include/mx.h.  bf16 arrays are
held as uint16 bit patterns."""
from __future__ import annotations

import math

import numpy as np

from ops_ref import EPS32, HALF_BF16, f64

NONE, RELU, RELU2, SILU, GELU, GELU_TANH = range(6)
SOFTMAX, SIGMOID = 0, 1
MOST = float(np.finfo(np.float32).max)

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ---- routing ------------------------------------------------------------------------


def _sum32(*v):
    with np.errstate(over="ignore"):
        out = v[0].astype(np.float32)
        for x in v[1:]:
            out = (out + x).astype(np.float32)
    return out


def route(x, score, bias, groups, topk_groups, group_best, topk, renorm, scale):
    """(ids, weights, bound) of logits x (float32 or float64 [T, E]); bias float32.

    Bound of a weight, relative, in half steps of fp32: the exponential is off by a
    last place (two) and its rounded argument adds |x - max|, the sum by as much and
    by at most ten additions, its reciprocal and a product two.  Over their sum: topk
    additions and a division, of values that far off; the scale one more."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    with np.errstate(invalid="ignore"):
        masked = ~(x > -np.inf)
    x = np.where(masked, -np.inf, np.minimum(x, MOST))
    top = np.max(x, axis=1, keepdims=True)
    top = np.where(top > -np.inf, top, 0.0)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        if score == SIGMOID:
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            e = np.exp(x - top)
            total = e.sum(1, keepdims=True)
            s = np.where(total > 0, e / np.where(total > 0, total, 1), 0.0)
    depth = np.where(masked, 0.0, np.minimum(top - x, 104.0)).max(1) if score == SOFTMAX else 0.0
    tol = 20 + 2 * depth + 2 * topk
    if bias is None:
        c = x
    else:
        b = bias.astype(np.float32)
        masked = masked | ~(b > -np.inf)[None]
        c = np.minimum(_sum32(s.astype(np.float32), np.broadcast_to(b, (T, E))), np.float32(MOST))
        c = np.where(masked, -np.inf, c.astype(np.float64))
    if groups > 1:
        by = np.sort(c.reshape(T, groups, -1), axis=2)[:, :, ::-1]
        near = by[:, :, 0] if group_best == 1 else \
            _sum32(by[:, :, 0].astype(np.float32), by[:, :, 1].astype(np.float32)).astype(np.float64)
        order = np.argsort(-near, axis=1, kind="stable")[:, :topk_groups]
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, order, True, axis=1)
        c = np.where(np.repeat(kept, E // groups, axis=1), c, -np.inf)
    order = np.argsort(-c, axis=1, kind="stable")[:, :topk]
    live = np.take_along_axis(c, order, 1) > -np.inf
    w = np.where(live, np.take_along_axis(s, order, 1), 0.0)
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)
    w = w * float(np.float32(scale))
    tol = np.broadcast_to(np.asarray(tol, np.float64).reshape(-1, 1), (T, 1))
    return np.where(live, order, -1).astype(np.int32), w, np.abs(w) * tol * EPS32 + 2.0 ** -125


# ---- the norms around a block ----------------------------------------------------------


def mean_scale(v, eps):
    return 1 / np.sqrt((v * v).mean(1, keepdims=True) + float(np.float32(eps)))


def stream(x, post, gate, gate_ids, res, alpha, offset, eps, fp32):
    """(s, bound) before s is rounded to its type: x bf16 bits, res bf16 bits or float32.

    p passes the mean's root (its sum has at most 8 * 16 + 6 + 3 additions, half of
    whose relative error reaches the root; a division, a root and a reciprocal), the
    weight's addition and three products: under 90 half steps; the last addition
    and the rounding to the type follow."""
    p = f64(x)
    off = float(np.float32(offset))
    if post is not None:
        p = p * mean_scale(p, eps) * (off + f64(post))
    if gate is not None:
        ids = np.zeros(len(p), np.int64) if gate_ids is None else gate_ids.astype(np.int64)
        live = (ids >= 0) & (ids < len(gate))
        p = np.where(live[:, None], p * f64(gate)[np.where(live, ids, 0)], 0.0)
    r = 0.0
    if res is not None:
        r = float(np.float32(alpha)) * (res.astype(np.float64) if fp32 else f64(res))
    s = r + p
    d = 90 * EPS32 * np.abs(p) + EPS32 * np.abs(s)
    return s, d + (EPS32 if fp32 else HALF_BF16) * (np.abs(s) + d)


def second_norm(s, weight, offset, eps):
    """(y, bound) of the stored s (float64 of its values): as the first norm, without
    the gate, and one bf16 rounding."""
    y = s * mean_scale(s, eps) * (float(np.float32(offset)) + f64(weight))
    return y, (HALF_BF16 + 90 * EPS32) * np.abs(y)


# ---- the linear's epilogue ---------------------------------------------------------------


def fn(kind, z):
    if kind == RELU:
        return np.maximum(z, 0.0)
    if kind == RELU2:
        return np.maximum(z, 0.0) ** 2
    with np.errstate(over="ignore"):
        if kind == SILU:
            return z / (1 + np.exp(-z))
        if kind == GELU:
            return 0.5 * z * _erfc(-z * math.sqrt(0.5))
        if kind == GELU_TANH:
            u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            return z / (1 + np.exp(-2 * u))
    return z


def _slope(kind, z, dz):
    """A bound of |f'| within dz of z."""
    if kind == RELU2:
        return 2 * (np.abs(z) + dz)
    return {NONE: 1.0, RELU: 1.0, SILU: 1.1}.get(kind, 1.13)


# f's own error, relative (the header's statement)
OF_FN = {NONE: 0.0, RELU: 0.0, RELU2: EPS32}


def product(a, w, mx8):
    """(z, bound) of a Wf^T.  MXFP8: the scaled matrix cores add eight neighbouring
    products in fixed point, at most 7 * 2^-13 of their sum of magnitudes off; either
    way at most K fp32 additions, each off by a step (2^-23) at most."""
    K = a.shape[1]
    return a @ w.T, ((7 * 2.0 ** -13 if mx8 else 0.0) + K * 2.0 ** -23) * (np.abs(a) @ np.abs(w).T)


def epilogue(z, dz, bias, kind, gated, res):
    """(y, bound): the bias is one fp32 addition; f moves with its argument and has
    its own error; gate and residual are a product and an addition; one bf16 rounding."""
    if bias is not None:
        z = z + f64(bias)
        dz = dz + EPS32 * (np.abs(z) + dz)
    own = OF_FN.get(kind, 2.0 ** -14)
    g, dg = (z[:, 0::2], dz[:, 0::2]) if gated else (z, dz)
    h = fn(kind, g)
    d = _slope(kind, g, dg) * dg
    d = d + own * (np.abs(h) + d) + 2.0 ** -126 * (1 + np.abs(g))
    if gated:
        u, du = z[:, 1::2], dz[:, 1::2]
        d = d * (np.abs(u) + du) + np.abs(h) * du
        h = h * u
        d = d + EPS32 * (np.abs(h) + d)
    if res is not None:
        h = h + f64(res)
        d = d + EPS32 * (np.abs(h) + d)
    return h, d + HALF_BF16 * (np.abs(h) + d)
