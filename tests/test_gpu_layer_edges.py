"""Edges of the operators between a layer's products that need cases of their own:
gates and weights that are not finite, sums infinite or far out in an activation's
tails, and the forms of the products that only larger sizes reach."""
import numpy as np
import pytest

import layer_ref as ref
import ops_ref
import oracle
from test_gpu_layer import (BF16, MXFP8, NAN16, T16, Lin, bf16, block_inputs, check_block,  # noqa: F401
                            g, mx, rng, run_block)

pytestmark = pytest.mark.gpu

PINF16, NINF16 = 0x7F80, 0xFF80


# ---- the norms around a block -------------------------------------------------------


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("with_post", [False, True])
def test_block_norm_rows_without_a_gate(g, mx, with_post, fp32):
    """A row whose gate number is outside the gates is T(alpha * residual) whatever
    the gates, the post weight and x hold, and so are its y and its bytes."""
    r = rng(80, with_post, fp32)
    for M, K in ((14, 160), (5, 4096)):
        i = block_inputs(r, M, K, fp32, gates=3)
        out = [0, 3, 4] if M == 5 else [0, 3, 5, 9]
        i["gids"][:] = 1 + np.arange(M) % 2
        i["gids"][out] = (-1, 3, 2 ** 31 - 1, -2 ** 31)[:len(out)]
        i["gate"][0] = (PINF16, NINF16, 0x7FC0, 0x3F80) * (K // 4)
        i["x"][out[1]] = NAN16
        for post in ([i["post"], (0, PINF16), (K - 1, 0x7FC0)] if with_post else [None]):
            if isinstance(post, tuple):
                at, bits = post
                post = i["post"].copy()
                post[at] = bits
            for res in (i["res"], None):
                a = (i["x"], post, i["gate"], i["gids"], res, 0.75, i["w"], 0.0, 1e-6, MXFP8, 0, fp32)
                got = run_block(g, mx, *a)
                rows = lambda v: None if v is None else v[out]                       # noqa: E731
                # against a call in which gates, weight and x are ordinary
                check_block([rows(v) for v in got], np.full_like(i["x"][out], 0x3F80), i["post"],
                            np.full_like(i["gate"], 0x3F80), i["gids"][out], rows(res), *a[5:])


# ---- the linear's epilogue -----------------------------------------------------------


FORMS = [  # elem, layout, M, N, K, act, form: every kernel with an epilogue
    (0, 0, 3, 64, 96, BF16, "x"), (1, 0, 4, 64, 4096, BF16, "x"),
    (0, 1, 16, 64, 1024, MXFP8, "x"), (0, 0, 5, 64, 1024, MXFP8, "x"), (0, 1, 9, 64, 1568, MXFP8, "x"),
    (0, 0, 9, 64, 1024, MXFP8, "given"), (0, 1, 9, 64, 1024, MXFP8, "t16"),
    (0, 0, 6, 64, 8224, MXFP8, "x"),
    (0, 1, 70, 64, 160, MXFP8, "t16"), (0, 0, 1025, 3600, 160, MXFP8, "t16"),
    (0, 1, 2100, 3616, 160, MXFP8, "t16")]


def of_bias(g, elem, layout, M, N, K, act):
    """A product whose sums are the bias: x is zeros."""
    lin = Lin(g, rng(81, elem, layout, M, N, K), elem, layout, 1, N, K, act)
    lin.sizes, lin.x = (M, N, K), np.zeros((M, K), np.uint16)
    if act != BF16:
        lin.q, lin.c = oracle.quant_act(lin.x, 0)
    return lin


def values(bits):
    return ops_ref.f64(np.asarray(bits, np.uint16))


@pytest.mark.parametrize("elem,layout,M,N,K,act,form", FORMS)
def test_linear_epilogue_infinite_sums(g, mx, elem, layout, M, N, K, act, form):
    """An infinite sum gives the activation's limit (+inf, or 0 on the left), a NaN a
    NaN, the largest numbers themselves."""
    lin = of_bias(g, elem, layout, M, N, K, act)
    z16 = np.resize(np.array([PINF16, NINF16, 0x7FC0, 0x7F7F, 0xFF7F, 0x6000, 0xE000, 0x3F80],
                             np.uint16), N)
    z = values(z16)
    for kind in range(6):
        with np.errstate(invalid="ignore", over="ignore"):
            want = ref.fn(kind, np.where(np.isfinite(z), z, 1.0))
        if kind != ref.NONE:
            want = np.where(z == -np.inf, 0.0, want)
        else:
            want = np.where(z == -np.inf, z, want)
        want = np.where(z == np.inf, z, np.where(np.isnan(z), z, want))
        y = values(lin.run(mx, form, z16, kind, False, None))
        # the gate's partners are 2 and 3 in turn: z stands at the even rows
        paired = np.stack([z16[:N // 2], np.resize(np.array([0x4000, 0xC040], np.uint16), N // 2)], 1)
        yg = values(lin.run(mx, form, np.ascontiguousarray(paired).reshape(-1), kind, True, None))
        for got, exact in ((y, want), (yg, want[:N // 2] * np.resize([2.0, -3.0], N // 2))):
            exact = np.broadcast_to(exact, got.shape)
            big = np.isinf(exact) | (np.abs(exact) > 2.0 ** 128 * (1 - 2.0 ** -9))
            near = np.where(big | np.isnan(exact), 0.0, exact)
            assert np.array_equal(np.isnan(got), np.isnan(exact)), kind
            assert np.array_equal(got[big], np.sign(exact[big]) * np.inf), kind
            err = np.abs(np.where(big | np.isnan(exact), 0.0, got) - near)
            assert (err <= (2.0 ** -8 + 2.0 ** -13) * np.abs(near) + 2.0 ** -126).all(), kind


@pytest.mark.parametrize("elem,layout,M,N,K,act,form", [f for f in FORMS if f[2] < 100])
def test_linear_epilogue_tails(g, mx, elem, layout, M, N, K, act, form):
    """f within 2^-14 of its value, relative, down to 2^-126, and one bf16 rounding: at
    every bf16 number from -4 to -128 and at small ones."""
    small = (0x0080 + 64 * np.arange(96)) | np.array([[0], [0x8000]])           # from 2^-126
    z16 = np.concatenate([np.arange(0xC080, 0xC300), small.reshape(-1)]).astype(np.uint16)
    N = (len(z16) + 31) // 32 * 32
    z16 = np.resize(z16, N)
    lin = of_bias(g, elem, layout, M, N, K, act)
    z = values(z16)
    for kind in (ref.SILU, ref.GELU, ref.GELU_TANH):
        want = ref.fn(kind, z)
        y = values(lin.run(mx, form, z16, kind, False, None))
        of_f = np.where(np.abs(want) >= 2.0 ** -126, 2.0 ** -14 * np.abs(want), 2.0 ** -126)
        err = np.abs(y - want)
        bad = err > of_f + 2.0 ** -8 * (np.abs(want) + of_f)
        assert not bad.any(), (kind, z[bad.any(0)][:8], y[bad][:8])


# Sizes that reach a kernel's larger forms: layout, M, N, K, act, form, the kernel and the
# end of its plan in the dispatch trace (tests/test_layer_trace_cpu.py holds them to it).
LARGER = [
    # K that the wavefronts do not share evenly, four tiles a workgroup
    (0, 64, 4096, 96, MXFP8, "x", "gemv_w8_kernel", "1 waves x 1 steps x 4 tiles"),
    (0, 64, 4160, 160, MXFP8, "x", "gemv_w8_kernel", "2 waves x 1 steps x 4 tiles"),
    (1, 17, 7200, 608, MXFP8, "given", "gemv_w8_kernel", "5 waves x 1 steps x 4 tiles"),
    (0, 64, 4096, 1568, MXFP8, "x", "gemv_w8_kernel", "8 waves x 2 steps x 4 tiles"),
    (1, 50, 4128, 1568, MXFP8, "given", "gemv_w8_kernel", "8 waves x 2 steps x 4 tiles"),
    (0, 49, 4144, 1536, T16, "t16", "gemv_w8_kernel", "8 waves x 2 steps x 4 tiles"),
    (1, 16, 14336, 1536, MXFP8, "given", "gemv_w8_kernel", "8 waves x 2 steps x 4 tiles"),
    # even K, four tiles a workgroup
    (0, 64, 4096, 1024, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 1 steps x 4 tiles"),
    (1, 40, 6144, 2048, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 2 steps x 4 tiles"),
    (1, 64, 4096, 4096, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 4 steps x 4 tiles"),
    (0, 50, 4096, 4096, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 4 steps x 4 tiles"),
    (0, 50, 2112, 7168, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 7 steps x 4 tiles"),
    (0, 49, 2112, 7168, MXFP8, "x", "gemv_w8_fused_kernel", "8 waves x 7 steps x 4 tiles"),
    (1, 64, 4096, 2048, T16, "t16", "gemv_w8_even_kernel", "8 waves x 2 steps x 4 tiles"),
    (0, 61, 4096, 4096, T16, "t16", "gemv_w8_even_kernel", "8 waves x 4 steps x 4 tiles"),
    (0, 50, 4096, 1024, MXFP8, "given", "gemv_w8_rm_kernel", "8 waves x 1 steps x 4 tiles"),
    # prefill, whole steps of K: tiles of 128, 224 and 256 weight rows, eight steps an
    # iteration and a remainder
    (0, 1025, 3600, 1024, T16, "t16", "gemm_w8a8_kernel", "128 x 256 tiles"),
    (1, 1025, 3616, 1152, MXFP8, "x", "gemm_w8a8_kernel", "128 x 256 tiles"),
    (0, 1800, 5376, 1024, T16, "t16", "gemm_w8a8_kernel", "224 x 256 tiles"),
    (1, 1800, 5376, 1152, MXFP8, "x", "gemm_w8a8_kernel", "224 x 256 tiles"),
    (1, 2500, 4064, 1024, T16, "t16", "gemm_w8a8_kernel", "256 x 256 tiles"),
    (0, 2500, 4064, 1152, MXFP8, "given", "gemm_w8a8_kernel", "256 x 256 tiles"),
    (1, 2500, 4064, 1152, MXFP8, "x", "gemm_w8a8_kernel", "256 x 256 tiles")]


@pytest.mark.parametrize("layout,M,N,K,act,form,kernel,plan", LARGER)
def test_linear_epilogue_larger_forms(g, mx, layout, M, N, K, act, form, kernel, plan):
    r = rng(82, layout, M, N, K)
    lin = Lin(g, r, 0, layout, M, N, K, act, rule=M % 2)
    cases = [(ref.SILU, True, False, True), (ref.NONE, False, True, True),
             (ref.GELU_TANH, False, True, False)]
    if M <= 64:                          # (the definition's erfc takes its time)
        cases.append((ref.GELU, True, True, True))
    for n, (kind, gated, with_bias, with_res) in enumerate(cases):
        bias = bf16(r, N) if with_bias else None
        res = bf16(r, M, N // 2 if gated else N, scale=2) if with_res else None
        y = lin.run(mx, form, bias, kind, gated, res, pad=8 * n)
        out, tol = ref.epilogue(lin.z, lin.dz, bias, kind, gated, res)
        ops_ref.assert_within(y, out, tol, f"fn {kind} gated {gated}")
        if with_res:
            assert np.array_equal(lin.run(mx, form, bias, kind, gated, res, pad=8 * n, inplace=True), y)
