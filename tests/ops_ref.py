"""Plain 64-bit definitions of the operators around the linear, for the tests:
numpy only, written from the formulas of include/mx.h.  bf16 arrays are held
as uint16 bit patterns."""
from __future__ import annotations

import numpy as np

from microscaling_quantized_linear_amd import workloads as wl

HALF_BF16 = 2.0 ** -8           # half a bf16 step, relative to the value
EPS32 = 2.0 ** -24              # half an fp32 step


def f64(bits: np.ndarray) -> np.ndarray:
    return wl.bf16_bits_to_f32(bits).astype(np.float64)


def e4m3_table() -> np.ndarray:
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8), 2.0 ** -6 * m / 8)
    return np.where(b >= 128, -v, v)


def e2m1_table() -> np.ndarray:
    v = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.concatenate([v, -v])


def pow2(codes: np.ndarray) -> np.ndarray:
    return 2.0 ** (codes.astype(np.float64) - 127)


def weights(elem, layout, E, N, K, w, codes) -> np.ndarray:
    """[E, N, K] from standard bytes and codes."""
    if elem == 0:
        v = e4m3_table()[w.reshape(E, N, K)]
    else:
        b = w.reshape(E, N, K // 2)
        v = np.stack([e2m1_table()[b & 15], e2m1_table()[b >> 4]], -1).reshape(E, N, K)
    s = pow2(codes).reshape(E, -1, K // 32)
    if layout == 1:
        s = np.repeat(s, 32, axis=1)
    return (v.reshape(E, N, K // 32, 32) * s[..., None]).reshape(E, N, K)


def activations(q, c) -> np.ndarray:
    """[M, K] from e4m3 bytes and E8M0 codes."""
    M, K = q.shape
    return (e4m3_table()[q].reshape(M, K // 32, 32) * pow2(c)[..., None]).reshape(M, K)


def residual_sum(x, res):
    """bf16 bits of x + res: one fp32 addition, rounded to bf16."""
    if res is None:
        return x
    return wl.f32_to_bf16_bits(wl.bf16_bits_to_f32(x) + wl.bf16_bits_to_f32(res))


def rms_norm(s, weight, eps):
    v = f64(s)
    return v / np.sqrt((v * v).mean(1, keepdims=True) + float(np.float32(eps))) * f64(weight)


def sort(ids, E):
    """(offsets, rows, pos) of routed ids [T, topk]."""
    T, topk = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    live = key[order] < E
    rows = np.where(live, order // topk, -1).astype(np.int32)
    pos = np.empty(T * topk, np.int32)
    pos[order] = np.where(live, np.arange(T * topk), -1)
    return offsets, rows, pos.reshape(T, topk)


def grouped(a, w, offsets, epi):
    """(result, bound): the fp64 products of rows [offsets[e], offsets[e + 1])
    with w[e], zeros elsewhere, and how far a kernel may be off:
    * the scaled matrix cores add the products of eight neighbouring K values in
      fixed point, whose last place is 2^-13 of the binade of the group's largest
      exponent sum (measured: beside 2^16 and -2^16 a product of 2^3 survives, one
      of 2^2 does not; in the next group of eight it does.  e2m1 weights: 2^-3
      beside 2^10, not 2^-4).  The largest product, of two 4-bit significands, is
      exact; each of the other seven loses less than a last place, at most 2^-13
      of the largest, so a group is off by at most 7 * 2^-13 of its sum of
      magnitudes;
    * at most K additions of group sums in fp32, each off by at most a step (2^-23)
      of the sum of magnitudes;
    * one bf16 rounding.
    SiLU: |silu'| <= 1.1; its exponential is taken of an argument rounded to fp32,
    so off by |g| 2^-23 relative, plus 2^-20 for the function, the division and
    the products."""
    M, K = a.shape
    E, N, _ = w.shape
    out = np.zeros((M, N // 2 if epi else N))
    tol = np.zeros_like(out)
    for e in range(E):
        r = slice(max(0, int(offsets[e])), min(M, int(offsets[e + 1])))
        if r.start >= r.stop:
            continue
        z = a[r] @ w[e].T
        d = (7 * 2.0 ** -13 + K * 2.0 ** -23) * (np.abs(a[r]) @ np.abs(w[e]).T)
        if epi:
            g, u, dg, du = z[:, 0::2], z[:, 1::2], d[:, 0::2], d[:, 1::2]
            sg = g / (1 + np.exp(np.minimum(-g, 700.0)))
            out[r] = sg * u
            d = 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du
            d = d + np.abs(out[r]) * (2.0 ** -20 + np.abs(g) * 2.0 ** -23)
        else:
            out[r] = z
        tol[r] = d + HALF_BF16 * (np.abs(out[r]) + d)
    return out, tol


def combine(ys, pos, wts):
    """(result, bound): topk fp32 multiply-adds, one bf16 rounding."""
    v = f64(ys)
    live = (pos >= 0) & (pos < len(ys))
    w = np.where(live, wts.astype(np.float64), 0.0)
    g = np.where(live[..., None], v[np.where(live, pos, 0)], 0.0)
    out = np.einsum("tk,tkn->tn", w, g)
    mag = np.einsum("tk,tkn->tn", np.abs(w), np.abs(g))
    d = (pos.shape[1] + 1) * EPS32 * mag
    return out, d + HALF_BF16 * (np.abs(out) + d)


def lora(x, a, b, scales, ids, base):
    """(result, bound).  v = scale x A^T: K fp32 additions, each off by at most a
    step (2^-23) of the sum of magnitudes, then a scale (one rounding); held as
    two bf16 numbers, off by 2^-16 relative; against B another R products (of both
    numbers) in fp32; base added and rounded once."""
    L, R, K = a.shape
    out = f64(base)
    tol = np.zeros_like(out)
    for g in range(L):
        m = ids == g
        if not m.any():
            continue
        s = 1.0 if scales is None else float(scales[g])
        xa, A, B = f64(x[m]), f64(a[g]), f64(b[g])
        v = s * (xa @ A.T)
        dv = abs(s) * K * 2.0 ** -23 * (np.abs(xa) @ np.abs(A).T)
        dv = dv + (2.0 ** -16 + 2.0 ** -23) * (np.abs(v) + dv)
        d = v @ B.T
        tol[m] = dv @ np.abs(B).T + 2 * R * 2.0 ** -23 * ((np.abs(v) + dv) @ np.abs(B).T)
        out[m] = out[m] + d
    tol += EPS32 * np.abs(out)
    live = (ids >= 0) & (ids < L)
    tol = np.where(live[:, None], tol + HALF_BF16 * (np.abs(out) + tol), 0.0)
    return out, tol


def assert_within(bits, ref, tol, what=""):
    """Every bf16 value within its bound of the reference (2^-133, half the
    smallest bf16 subnormal, on top)."""
    err = np.abs(f64(bits).reshape(ref.shape) - ref)
    bad = ~(err <= tol + 2.0 ** -133)
    assert not bad.any(), (
        f"{what}: {bad.sum()} of {bad.size} values beyond their bound; first at "
        f"{tuple(int(i) for i in np.argwhere(bad)[0])}, worst ratio "
        f"{np.nanmax(err[bad] / (tol[bad] + 2.0 ** -133)):.3g}")
