"""The operators between a layer's products on the GPU -- the choice of experts,
the norms around a block with gate and residual scale, the linear with
activation and residual in its epilogue -- against their plain 64-bit
definitions (tests/layer_ref.py), at the sizes, strides, masks and orders where
they could go wrong, alone and run together."""
import numpy as np
import pytest

import layer_ref as ref
import ops_ref
import oracle
from microscaling_quantized_linear_amd import workloads as wl

pytestmark = pytest.mark.gpu

BF16, MXFP8, T16 = 0, 1, 2
NAN16 = 0x7FC1                 # a bf16 NaN that no output holds
INF = float("inf")


@pytest.fixture(scope="module")
def g():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxgpu
    return mxgpu


@pytest.fixture(scope="module")
def mx(g):
    import microscaling_quantized_linear_amd
    return microscaling_quantized_linear_amd


def rng(*key):
    return np.random.default_rng([91, *key])


def bf16(r, *shape, scale=1.0):
    return wl.f32_to_bf16_bits(r.standard_normal(shape).astype(np.float32) * np.float32(scale))


def strided(g, a, ld):
    """A device buffer [rows, ld] with `a` in its first columns, NaN behind."""
    buf = np.full((a.shape[0], ld), NAN16 if a.dtype == np.uint16 else np.nan, a.dtype)
    buf[:, :a.shape[1]] = a
    return g.dev(buf)


def out16(g, rows, ld):
    import torch
    return torch.full((rows, ld), NAN16, dtype=torch.int16, device=g.DEV)


def bytes_(g, *shape, fill=0xAB):
    import torch
    return torch.full(shape, fill, dtype=torch.uint8, device=g.DEV)


# ---- the choice of experts -----------------------------------------------------------


def run_route(g, mx, x, score, bias=None, groups=1, keep=1, best=1, topk=2, renorm=True, scale=1.0,
              pad=0, shift=0, stream=None):
    """x: float32, or uint16 bf16 bits [T, E].  shift: elements before the first."""
    import torch
    T, E = x.shape
    ld = E + pad
    buf = np.full(shift + T * ld, np.nan if x.dtype == np.float32 else NAN16, x.dtype)
    v = buf[shift:].reshape(T, ld)
    v[:, :E] = x
    d = g.dev(buf)
    ids = torch.full((T * topk + 1,), -7, dtype=torch.int32, device=g.DEV)
    w = torch.full((T * topk + 1,), -7.0, dtype=torch.float32, device=g.DEV)
    mx.mx_moe_route(E, T, topk, 1 if x.dtype == np.float32 else 0,
                    d.data_ptr() + shift * x.dtype.itemsize, ld, score,
                    None if bias is None else g.dev(bias), groups, keep, best, renorm, scale, ids, w,
                    stream)
    torch.cuda.synchronize()
    assert int(ids[-1]) == -7 and float(w[-1]) == -7.0
    return ids[:-1].cpu().numpy().reshape(T, topk), w[:-1].cpu().numpy().reshape(T, topk)


def check_route(got, x, score, bias=None, groups=1, keep=1, best=1, topk=2, renorm=True, scale=1.0):
    v = x if x.dtype == np.float32 else wl.bf16_bits_to_f32(x)
    ids, w, tol = ref.route(v, score, bias, groups, keep, best, topk, renorm, scale)
    assert np.array_equal(got[0], ids)
    err = np.abs(got[1].astype(np.float64) - w)
    assert (err <= tol).all(), float((err / tol).max())


ROUTES = [  # E, T, topk, groups, keep, best
    (1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 1, 1), (8, 1, 2, 1, 1, 1), (32, 16, 8, 1, 1, 1),
    (32, 2000, 8, 8, 3, 2), (60, 5, 4, 1, 1, 1), (64, 1500, 6, 8, 3, 2), (65, 70, 9, 5, 2, 2),
    (128, 1100, 8, 1, 1, 1), (160, 9, 6, 8, 3, 1), (160, 1300, 6, 8, 3, 1), (256, 1, 8, 8, 4, 2),
    (256, 1025, 8, 8, 4, 2), (256, 40, 64, 64, 32, 2), (255, 33, 17, 3, 2, 1), (257, 50, 8, 1, 1, 1),
    (384, 1200, 8, 1, 1, 1), (510, 20, 10, 51, 7, 2), (512, 300, 8, 16, 4, 2),
    (1000, 17, 10, 8, 4, 2), (1024, 130, 64, 64, 40, 1), (72, 1030, 64, 1, 1, 1),
    (31, 1029, 31, 1, 1, 1)]


@pytest.mark.parametrize("E,T,topk,groups,keep,best", ROUTES)
def test_route(g, mx, E, T, topk, groups, keep, best):
    r = rng(1, E, T)
    base = (1.5 * r.standard_normal((T, E)) + 0.7 * r.standard_normal(E)).astype(np.float32)
    bias = (0.1 * r.standard_normal(E)).astype(np.float32)
    half = wl.f32_to_bf16_bits(base)                     # many equal logits
    for score in (0, 1):
        for x, b, renorm, pad, shift in ((base, bias, True, 0, 0), (half, bias, False, 4, 4),
                                         (base, None, True, 3, 1), (half, None, False, 0, 0),
                                         (half, bias, True, 1, 1)):
            kw = dict(groups=groups, keep=keep, best=best if b is not None else 1, topk=topk,
                      renorm=renorm, scale=2.5 if renorm else 1.0)
            check_route(run_route(g, mx, x, score, b, pad=pad, shift=shift, **kw), x, score, b, **kw)


@pytest.mark.parametrize("E,T", [(32, 40), (256, 1100), (300, 30), (1024, 9)])
def test_route_masks(g, mx, E, T):
    """Masked experts, tokens with fewer experts than choices, tokens and groups with
    none, infinities, NaN; masked by the bias."""
    r = rng(2, E, T)
    x = r.standard_normal((T, E)).astype(np.float32)
    x[r.random((T, E)) < 0.3] = -INF
    x[r.random((T, E)) < 0.1] = np.nan
    x[0] = -INF
    x[1] = np.nan
    x[2, 1:] = -INF                                      # one expert left
    x[3, : E // 2] = -INF                                # groups without any
    x[4, 5] = INF
    x[5] = INF
    x[6, :4] = (INF, -INF, np.nan, -0.0)
    x[7] = -np.float32(ref.MOST)
    x[8] = 0.0
    x[8, ::3] = -0.0                                     # ties with 0
    bias = (0.1 * r.standard_normal(E)).astype(np.float32)
    bias[[3, 8]] = (-INF, np.nan)
    bias[11] = INF
    for score in (0, 1):
        for b in (None, bias):
            for groups, keep, best in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
                kw = dict(groups=groups, keep=keep, best=best if b is not None else 1, topk=6)
                got = run_route(g, mx, x, score, b, **kw)
                assert (got[0][:2] == -1).all() and (got[1][:2] == 0).all()
                check_route(got, x, score, b, **kw)


def test_route_wide_logits(g, mx):
    """Logits far apart: scores that round to 0 and 1, ties among them, weights of
    tiny scores."""
    r = rng(3)
    x = (40 * r.standard_normal((300, 128))).astype(np.float32)
    b = (0.01 * r.standard_normal(128)).astype(np.float32)
    for score in (0, 1):
        for bias in (None, np.zeros(128, np.float32), b):
            for renorm in (False, True):
                kw = dict(topk=5, renorm=renorm)
                check_route(run_route(g, mx, x, score, bias, **kw), x, score, bias, **kw)


def test_route_near_ties(g, mx):
    """Biased scores a last place apart: the order of the correctly rounded ones."""
    r = rng(4)
    T, E = 2000, 64
    s = 0.5 + np.float64(2.0) ** -24 * r.integers(0, 6, (T, E))
    x = np.log(s / (1 - s)).astype(np.float32)
    for bias in (np.zeros(E, np.float32), np.full(E, 0.25, np.float32)):
        check_route(run_route(g, mx, x, 1, bias, topk=8), x, 1, bias, topk=8)


@pytest.mark.parametrize("E,groups", [(64, 8), (96, 8), (256, 8), (256, 4), (128, 32)])
def test_route_near_tied_groups(g, mx, E, groups):
    """Groups whose scores are a last place apart, in every token or in a few of them:
    those of the correctly rounded scores are kept."""
    r = rng(5, E, groups)
    T = 1500
    s = 0.5 + np.float64(2.0) ** -24 * r.integers(0, 6, (T, E))
    x = np.log(s / (1 - s)).astype(np.float32)
    few = (1.5 * r.standard_normal((T, E))).astype(np.float32)
    few[::97] = x[::97]
    few[5::97, E // groups:] = -INF
    half = np.full(E, 0.25, np.float32)
    for v in (x, few):
        for score in (0, 1):
            for bias in (half, (0.1 * r.standard_normal(E)).astype(np.float32)):
                for best in (1, 2):
                    kw = dict(groups=groups, keep=groups // 2, best=best, topk=6)
                    check_route(run_route(g, mx, v, score, bias, **kw), v, score, bias, **kw)


def test_route_tokens_do_not_depend_on_the_call(g, mx):
    """A token alone, in a small call and in a large one (another form): the same bits."""
    for E in (24, 64, 100, 256, 512):
        r = rng(5, E)
        T = 3000
        x = r.standard_normal((T, E)).astype(np.float32)
        bias = (0.1 * r.standard_normal(E)).astype(np.float32)
        for score, b, renorm in ((0, None, True), (0, None, False), (0, bias, False), (1, bias, True)):
            big = run_route(g, mx, x, score, b, topk=4, renorm=renorm)
            for t0, t1 in ((0, 1), (7, 40), (2990, 3000)):
                part = run_route(g, mx, x[t0:t1], score, b, topk=4, renorm=renorm)
                assert np.array_equal(big[0][t0:t1], part[0])
                assert np.array_equal(big[1][t0:t1].view(np.uint32), part[1].view(np.uint32))


# ---- the norms around a block ----------------------------------------------------------


def run_block(g, mx, x, post, gate, gids, res, alpha, w, offset, eps, act, rule, fp32, keep=True,
              want_sum=True, pad=0, stream=None):
    """The call's outputs on the host: (sum, y, xq, xcodes), T16 buffers unpacked to
    padded row-major; checks that nothing outside the outputs changed."""
    import torch
    M, K = x.shape
    xd = strided(g, x, K + pad)
    rd = strided(g, res, K + 2 * pad) if res is not None else None
    gd = strided(g, gate, K + 3 * pad) if gate is not None else None
    if fp32:
        s = torch.full((M + 1, K + pad), -7.5, dtype=torch.float32, device=g.DEV)
    else:
        s = out16(g, M + 1, K + pad)
    s = s if want_sum else None
    y = out16(g, M + 1, K + 3 * pad) if w is not None and (keep or act == BF16) else None
    ldq = ldc = 0
    if act == T16:
        qb, cb = mx.mx_act_t16_sizes(M, K)
        q, c = bytes_(g, qb + 16), bytes_(g, cb + 16)
    else:
        ldq, ldc = K + 2 * pad, K // 32 + pad
        q, c = bytes_(g, M + 1, ldq), bytes_(g, M + 1, ldc)
    dev = lambda a: None if a is None else g.dev(a)                             # noqa: E731
    mx.mx_block_norm(M, K, xd, K + pad, dev(post), gd, 0 if gate is None else len(gate),
                     K + 3 * pad if gd is not None else 0, dev(gids), 1 if fp32 else 0, rd,
                     K + 2 * pad if rd is not None else 0, alpha, dev(w), offset, eps, act, rule, s,
                     K + pad if s is not None else 0, y, K + 3 * pad if y is not None else 0, q, ldq,
                     c, ldc, stream)
    torch.cuda.synchronize()
    hs = hy = hq = hc = None
    if s is not None:
        hs, canary = (s.cpu().numpy(), -7.5) if fp32 else (g.host_u16(s), NAN16)
        assert (hs[M:] == canary).all() and (hs[:, K:] == canary).all()
        hs = hs[:M, :K]
    if y is not None:
        hy = g.host_u16(y)
        assert (hy[M:] == NAN16).all() and (hy[:, K:] == NAN16).all()
        hy = hy[:M, :K]
    hq, hc = q.cpu().numpy(), c.cpu().numpy()
    if act == T16:
        assert (hq[qb:] == 0xAB).all() and (hc[cb:] == 0xAB).all()
        hq, hc = g.t16_unpack(hq[:qb], hc[:cb], M, K)
        assert (hq[M:] == 0).all() and (hq[:, K:] == 0).all()
        assert (hc[M:] == 127).all() and (hc[:, K // 32:] == 127).all()
        hq, hc = hq[:M, :K], hc[:M, :K // 32]
    elif act == MXFP8:
        assert (hq[M:] == 0xAB).all() and (hq[:, K:] == 0xAB).all()
        assert (hc[M:] == 0xAB).all() and (hc[:, K // 32:] == 0xAB).all()
        hq, hc = hq[:M, :K], hc[:M, :K // 32]
    else:
        assert (hq == 0xAB).all() and (hc == 0xAB).all()
    return hs, hy, hq, hc


def check_block(out, x, post, gate, gids, res, alpha, w, offset, eps, act, rule, fp32):
    """s against the definition, y against that of the stored s, the bytes against
    the quantization of y."""
    s, y, q, c = out
    want, tol = ref.stream(x, post, gate, gids, res, alpha, offset, eps, fp32)
    v = s.astype(np.float64) if fp32 else ops_ref.f64(s)
    err = np.abs(v - want)
    assert (err <= tol + 2.0 ** -133).all(), float((err / (tol + 2.0 ** -133)).max())
    if w is None:
        return
    if y is not None:
        exact, tol = ref.second_norm(v, w, offset, eps)
        ops_ref.assert_within(y, exact, tol, "second norm")
        if act != BF16:
            oq, oc = oracle.quant_act(y, rule)
            assert np.array_equal(c, oc) and np.array_equal(q, oq)


def block_inputs(r, M, K, fp32, gates=3, offset=0.0):
    vec = lambda: wl.f32_to_bf16_bits((1 - offset + 0.3 * r.standard_normal(K)).astype(np.float32))  # noqa: E731
    res = 3 * r.standard_normal((M, K)).astype(np.float32)
    return dict(x=bf16(r, M, K), post=vec(), gate=bf16(r, gates, K), w=vec(),
                gids=r.integers(0, gates, M).astype(np.int32),
                res=res if fp32 else wl.f32_to_bf16_bits(res))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("act", [BF16, MXFP8, T16])
@pytest.mark.parametrize("M,K,pad", [
    (1, 32, 0), (9, 32, 16), (1, 7168, 0), (3, 96, 16), (16, 512, 0), (17, 544, 32), (130, 1024, 0),
    (5, 1568, 16), (50, 1568, 0), (33, 4096, 0), (2, 4128, 16), (40, 7168, 16), (2, 8192, 0),
    (1, 16384, 0), (2, 20000 // 32 * 32, 16), (1, 32768, 0), (1, 65536, 0)])
def test_block_norm(g, mx, M, K, pad, act, fp32):
    r = rng(20, M, K, fp32)
    for n, (rule, post, gate, gids, res, alpha, offset) in enumerate((
            (0, True, True, True, True, 0.8, 0.0), (1, True, False, False, True, 1.0, 1.0),
            (0, False, True, False, True, -1.5, 0.0), (1, True, True, True, False, 2.0, 1.0))):
        i = block_inputs(r, M, K, fp32, offset=offset)
        a = (i["x"], i["post"] if post else None, i["gate"] if gate else None,
             i["gids"] if gids else None, i["res"] if res else None, alpha, i["w"], offset, 1e-6,
             act, rule, fp32)
        check_block(run_block(g, mx, *a, pad=pad), *a)


@pytest.mark.parametrize("fp32", [False, True])
def test_block_norm_outputs_left_out(g, mx, fp32):
    """No sum, no bf16 y: the bytes stay the same; no second norm: the same sum."""
    r = rng(21)
    M, K = 21, 1056
    i = block_inputs(r, M, K, fp32)
    for act in (MXFP8, T16):
        a = (i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.5)
        full = run_block(g, mx, *a, i["w"], 0.0, 1e-5, act, 0, fp32)
        bare = run_block(g, mx, *a, i["w"], 0.0, 1e-5, act, 0, fp32, keep=False, want_sum=False)
        assert bare[0] is None and bare[1] is None
        assert np.array_equal(full[2], bare[2]) and np.array_equal(full[3], bare[3])
        only = run_block(g, mx, *a, None, 0.0, 1e-5, BF16, 0, fp32)
        assert only[1] is None and np.array_equal(only[0], full[0])


def test_block_norm_is_add_rms_norm(g, mx):
    """Without post norm, gate and scale: the residual norm's sum exactly, its y within
    a rounding (the sums of squares differ in their order)."""
    import torch
    r = rng(22)
    M, K = 37, 7168
    i = block_inputs(r, M, K, False)
    s, y, _, _ = run_block(g, mx, i["x"], None, None, None, i["res"], 1.0, i["w"], 0.0, 1e-6, BF16, 0,
                           False)
    ys, ss = out16(g, M, K), out16(g, M, K)
    mx.mx_add_rms_norm(M, K, g.dev(i["x"]), K, g.dev(i["res"]), K, g.dev(i["w"]), 1e-6, BF16, 0, ss, K,
                       ys, K, None, 0, None, 0)
    torch.cuda.synchronize()
    assert np.array_equal(s, g.host_u16(ss))
    a, b = ops_ref.f64(y), ops_ref.f64(g.host_u16(ys))
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b)).all()


def test_block_norm_gate_numbers(g, mx):
    """Gate numbers outside the gates add nothing, also where x is NaN or infinite."""
    r = rng(23)
    M, K = 14, 160
    for fp32 in (False, True):
        i = block_inputs(r, M, K, fp32, gates=4)
        i["gids"][[0, 3, 5, 9]] = (-1, 4, 2 ** 31 - 1, -2 ** 31)
        i["x"][3] = NAN16
        i["x"][5, 7] = 0x7F80
        a = (i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.75, i["w"], 0.0, 1e-6, MXFP8, 0, fp32)
        out = run_block(g, mx, *a)
        clean = i["x"].copy()
        clean[[3, 5]] = 0x3F80
        check_block(out, clean, *a[1:])


def test_block_norm_rows_do_not_depend_on_the_call(g, mx):
    """A row alone, in a small call and in a large one: the same bits."""
    r = rng(24)
    for K in (64, 512, 1568, 7168):
        M = 700
        i = block_inputs(r, M, K, True)
        big = run_block(g, mx, i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.9, i["w"], 0.0, 1e-6,
                        T16, 0, True)
        for m0, m1 in ((0, 1), (5, 22), (698, 700)):
            part = run_block(g, mx, i["x"][m0:m1], i["post"], i["gate"], i["gids"][m0:m1],
                             i["res"][m0:m1], 0.9, i["w"], 0.0, 1e-6, T16, 0, True)
            for a, b in zip(big, part):
                assert np.array_equal(a[m0:m1].view(np.uint8), b.view(np.uint8))


def test_block_norm_ranges(g, mx):
    """Zero rows, tiny and large values, saturating blocks, zero gates and weights."""
    r = rng(25)
    M, K = 6, 128
    for fp32 in (False, True):
        i = block_inputs(r, M, K, fp32)
        i["x"][0] = 0
        i["x"][1] = bf16(r, K, scale=1e-18)
        i["x"][2] = bf16(r, K, scale=1e17)
        i["res"][:2] = 0
        i["w"][5], i["w"][6] = 0, 0x8000
        i["gate"][1] = 0
        for act in (MXFP8, T16):
            for rule in (0, 1):
                for eps in (0.5, 1e-12):
                    a = (i["x"], i["post"], i["gate"], i["gids"], i["res"], 1.0, i["w"], 0.0, eps, act,
                         rule, fp32)
                    check_block(run_block(g, mx, *a), *a)


@pytest.mark.parametrize("M,K", [(1, 64), (19, 7168), (130, 1568)])
def test_block_norm_in_place(g, mx, M, K):
    """sum on the residual, y on x (and the other way round): the separate call's values."""
    import torch
    r = rng(26, M, K)
    for fp32 in (False, True):
        i = block_inputs(r, M, K, fp32)
        s, y, _, _ = run_block(g, mx, i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.7, i["w"], 0.0,
                               1e-6, BF16, 0, fp32)
        for swap in ((False, True) if not fp32 else (False,)):
            xd, rd = g.dev(i["x"]), g.dev(i["res"])
            so, yo = (xd, rd) if swap else (rd, xd)
            mx.mx_block_norm(M, K, xd, K, g.dev(i["post"]), g.dev(i["gate"]), 3, K, g.dev(i["gids"]),
                             1 if fp32 else 0, rd, K, 0.7, g.dev(i["w"]), 0.0, 1e-6, BF16, 0, so, K, yo, K,
                             None, 0, None, 0)
            torch.cuda.synchronize()
            assert np.array_equal(so.cpu().numpy().view(s.dtype), s)
            assert np.array_equal(g.host_u16(yo), y)


# ---- the linear with an epilogue ----------------------------------------------------------


def weight(g, r, elem, layout, N, K, lo=118, hi=126):
    w = wl.e4m3_bytes(r, (1, N, K)) if elem == 0 else wl.fp4_bytes(r, (1, N, K // 2))
    codes = wl.codes(r, (N // (32 if layout else 1), K // 32), lo, hi)
    return ops_ref.weights(elem, layout, 1, N, K, w, codes)[0], g.pack(elem, layout, 1, N, K, w, codes)


class Lin:
    """One product: its inputs in every form, and its exact sums."""

    def __init__(self, g, r, elem, layout, M, N, K, act, rule=0):
        self.g, self.sizes, self.elem, self.layout, self.act, self.rule = g, (M, N, K), elem, layout, act, rule
        scale = 2.0 ** -4 * K ** -0.5                    # sums of a few units
        self.W, self.packed = weight(g, r, elem, layout, N, K)
        self.x = wl.f32_to_bf16_bits(
            wl.bf16_bits_to_f32(wl.activations(r, (M, K), 0.01)) * np.float32(scale))
        if act == BF16:
            self.a = ops_ref.f64(self.x)
        else:
            self.q, self.c = oracle.quant_act(self.x, rule)
            self.a = ops_ref.activations(self.q, self.c)
        self.z, self.dz = ref.product(self.a, self.W, act != BF16)

    def run(self, mx, form, bias, fn, gated, res, pad=0, inplace=False, rows=None, stream=None):
        import torch
        M, N, K = self.sizes
        x, sl = self.x, slice(None)
        if rows is not None:
            sl = rows
            x = x[sl]
            M = len(x)
        g, width = self.g, N // 2 if gated else N
        act, kw = self.act, dict(x=None, ldx=0, q=None, ldq=0, c=None, ldc=0)
        if form == "t16":
            act = T16
            kw["q"], kw["c"] = g.quant_t16(np.ascontiguousarray(x), self.rule)
        elif form == "given":
            ldq = (K + 15) // 16 * 16 + pad * 2
            buf = np.full((M, ldq), 0x7F, np.uint8)
            buf[:, :K] = self.q[sl]
            cb = np.full((M, K // 32 + 3), 0xFF, np.uint8)
            cb[:, :K // 32] = self.c[sl]
            kw.update(q=g.dev(buf), ldq=ldq, c=g.dev(cb), ldc=K // 32 + 3)
        else:
            kw.update(x=strided(g, x, K + pad), ldx=K + pad)
        need = mx.mx_linear_workspace(self.elem, self.layout, N, K, M, act, form != "x")
        ws = bytes_(g, max(need, 16), fill=0x7F)
        ldr, ldy = (width + 7) // 8 * 8 + pad, (width + 7) // 8 * 8 + 2 * pad
        rd = None
        if res is not None:
            buf = np.full((M + 1, ldr), NAN16, np.uint16)
            buf[:M, :width] = res[sl]
            rd = g.dev(buf)
        y = rd if inplace else out16(g, M + 1, ldy)
        mx.mx_linear_epilogue(self.elem, self.layout, N, K, *self.packed, M, act, self.rule, kw["x"],
                              kw["ldx"], kw["q"], kw["ldq"], kw["c"], kw["ldc"],
                              None if bias is None else g.dev(bias), fn, gated, rd,
                              ldr if rd is not None else 0, y, ldr if inplace else ldy,
                              ws if need else None, need, stream)
        torch.cuda.synchronize()
        h = g.host_u16(y)
        assert (h[M:] == NAN16).all() and (h[:, width:] == NAN16).all()
        return h[:M, :width]


LINEAR = [  # elem, layout, M, N, K, act, form
    # bf16 activations, at every launch shape of the GEMV
    (0, 0, 1, 16, 32, BF16, "x"), (0, 0, 3, 48, 96, BF16, "x"), (0, 1, 16, 96, 512, BF16, "x"),
    (0, 0, 8, 80, 1568, BF16, "x"), (0, 1, 17, 64, 2080, BF16, "x"), (0, 0, 5, 48, 4128, BF16, "x"),
    (1, 0, 2, 16, 32, BF16, "x"), (1, 0, 33, 48, 288, BF16, "x"), (1, 0, 4, 176, 1056, BF16, "x"),
    (1, 0, 7, 32, 3200, BF16, "x"), (1, 0, 4, 80, 4096, BF16, "x"), (1, 0, 90, 64, 544, BF16, "x"),
    # MXFP8, decode: quantized inside the kernel, ahead of it, given, T16
    (0, 1, 16, 64, 1024, MXFP8, "x"), (0, 0, 4, 96, 2048, MXFP8, "x"), (0, 1, 21, 64, 7168, MXFP8, "x"),
    (0, 0, 33, 4096, 1024, MXFP8, "x"), (0, 1, 16, 64, 8192, MXFP8, "x"), (0, 0, 32, 16, 4096, MXFP8, "x"),
    (0, 0, 3, 48, 160, MXFP8, "x"), (0, 1, 40, 96, 1568, MXFP8, "x"), (0, 1, 5, 7168, 1536, MXFP8, "x"),
    (0, 0, 9, 64, 1024, MXFP8, "given"), (0, 1, 18, 96, 7168, MXFP8, "given"),
    (0, 0, 3, 80, 1568, MXFP8, "given"), (0, 0, 9, 64, 1024, MXFP8, "t16"),
    (0, 1, 64, 96, 4096, MXFP8, "t16"), (0, 0, 2, 112, 608, MXFP8, "t16"),
    # K beyond the T16 GEMV's registers
    (0, 0, 6, 48, 8224, MXFP8, "x"), (0, 1, 18, 32, 8448, MXFP8, "given"),
    # prefill
    (0, 0, 65, 16, 32, MXFP8, "x"), (0, 1, 130, 288, 544, MXFP8, "x"), (0, 0, 300, 272, 1024, MXFP8, "given"),
    (0, 1, 257, 1792, 640, MXFP8, "t16"), (0, 0, 100, 1792, 1568, MXFP8, "x"),
    (0, 1, 70, 320, 2208, MXFP8, "t16"), (0, 0, 513, 240, 96, MXFP8, "x"), (0, 0, 66, 3584, 384, MXFP8, "x"),
    # more than a tile of 64 or of 128 weight rows for each compute unit
    (0, 0, 1025, 3600, 160, MXFP8, "t16"), (0, 1, 2100, 3616, 1056, MXFP8, "x"),
    (0, 0, 1800, 5376, 160, MXFP8, "x"), (0, 1, 2500, 4064, 1184, MXFP8, "given")]


@pytest.mark.parametrize("elem,layout,M,N,K,act,form", LINEAR)
def test_linear_epilogue(g, mx, elem, layout, M, N, K, act, form):
    r = rng(40, elem, layout, M, N, K)
    lin = Lin(g, r, elem, layout, M, N, K, act, rule=M % 2)
    for n, kind in enumerate(range(6)):
        for gated in (False, True):
            width = N // 2 if gated else N
            bias = bf16(r, N) if (n + gated) % 2 else None
            res = bf16(r, M, width, scale=2) if (n // 2 + gated) % 2 else None
            pad = 8 * (n % 3)
            y = lin.run(mx, form, bias, kind, gated, res, pad=pad)
            out, tol = ref.epilogue(lin.z, lin.dz, bias, kind, gated, res)
            ops_ref.assert_within(y, out, tol, f"fn {kind} gated {gated}")
            if res is not None:
                assert np.array_equal(
                    lin.run(mx, form, bias, kind, gated, res, pad=pad, inplace=True), y)


def test_linear_without_epilogue_is_mx_linear(g, mx):
    """No activation, gate or residual: mx_linear's bits; forms of one activation agree."""
    for elem, layout, M, N, K, act in ((0, 0, 5, 64, 1024, MXFP8), (0, 1, 200, 320, 544, MXFP8),
                                       (0, 0, 9, 96, 1568, BF16), (1, 0, 4, 80, 4096, BF16)):
        r = rng(41, M, N)
        lin = Lin(g, r, elem, layout, M, N, K, act)
        bias = bf16(r, N)
        want = g.linear(elem, layout, N, K, *lin.packed, act, x=lin.x, bias=bias)
        assert np.array_equal(lin.run(mx, "x", bias, 0, False, None), want)
        if act == MXFP8:
            res = bf16(r, M, N // 2)
            y = [lin.run(mx, f, bias, ref.SILU, True, res) for f in ("x", "given", "t16")]
            assert np.array_equal(y[0], y[1]) and np.array_equal(y[0], y[2])


@pytest.mark.parametrize("layout,M,N", [(0, 64, 2112), (1, 50, 2112), (0, 61, 2080), (1, 49, 2176)])
def test_linear_epilogue_more_than_one_round(g, mx, layout, M, N):
    """The GEMV that quantizes inside at more workgroups than compute units: four tiles
    a workgroup (two where the tiles do not divide), whole and partial token tiles.
    Without an epilogue the bits are mx_linear's."""
    K = 7168
    r = rng(43, layout, M, N)
    lin = Lin(g, r, 0, layout, M, N, K, MXFP8, rule=M % 2)
    for n, (kind, gated) in enumerate(((ref.SILU, True), (ref.GELU, False), (ref.NONE, False),
                                       (ref.RELU2, True))):
        bias = bf16(r, N) if n % 2 else None
        res = bf16(r, M, N // 2 if gated else N, scale=2) if n else None
        y = lin.run(mx, "x", bias, kind, gated, res, pad=8 * n)
        out, tol = ref.epilogue(lin.z, lin.dz, bias, kind, gated, res)
        ops_ref.assert_within(y, out, tol, f"fn {kind} gated {gated}")
        if res is not None:
            assert np.array_equal(lin.run(mx, "x", bias, kind, gated, res, pad=8 * n, inplace=True), y)
    bias = bf16(r, N)
    want = g.linear(0, layout, N, K, *lin.packed, MXFP8, x=lin.x, bias=bias, rule=M % 2)
    assert np.array_equal(lin.run(mx, "x", bias, 0, False, None), want)


def test_linear_epilogue_values(g, mx):
    """Sums over the whole range of the activations, far tails and beyond bf16 among
    them: a one-hot x hands z to each function exactly."""
    N, K = 64, 64
    z = np.concatenate([np.linspace(-20, 20, 2 * N), 2.0 ** np.linspace(-40, 40, N),
                        -(2.0 ** np.linspace(-40, 7, N))])
    # weights 1 on the diagonal; x holds the values
    w = np.zeros((1, N, K), np.uint8)
    w[0, np.arange(N), np.arange(N)] = 0x38                      # e4m3 1.0
    codes = np.full((N, K // 32), 127, np.uint8)
    packed = g.pack(0, 0, 1, N, K, w, codes)
    for M in (4, 80):
        x = np.resize(wl.f32_to_bf16_bits(z.astype(np.float32)), (M, K))
        lin = Lin.__new__(Lin)
        lin.g, lin.sizes, lin.elem, lin.layout, lin.act, lin.rule = g, (M, N, K), 0, 0, BF16, 0
        lin.packed, lin.x = packed, x
        for kind in range(6):
            y = lin.run(mx, "x", None, kind, False, None)
            out, tol = ref.epilogue(ops_ref.f64(x), np.zeros((M, N)), None, kind, False, None)
            ops_ref.assert_within(y, out, tol, f"fn {kind}")
    # the prefill kernel, with values that its activations hold exactly
    v = np.array([s * m * 2.0 ** e for s in (-1, 1) for m in (1, 1.25, 1.75)
                  for e in range(-24, 7)])
    M = 80
    x = np.zeros((M, K), np.uint16)
    x[:, 0::32] = np.resize(wl.f32_to_bf16_bits(v.astype(np.float32)), (M, K // 32))
    lin.sizes, lin.act, lin.x = (M, N, K), MXFP8, x
    for kind in range(6):
        for form in ("x", "t16"):
            y = lin.run(mx, form, None, kind, False, None)
            out, tol = ref.epilogue(ops_ref.f64(x), np.zeros((M, N)), None, kind, False, None)
            ops_ref.assert_within(y, out, tol, f"prefill, fn {kind}")


def test_linear_epilogue_batch_invariant(g, mx):
    """With the mode on, a row's result does not depend on the rows beside it."""
    r = rng(43)
    lin = Lin(g, r, 0, 1, 200, 160, 1568, MXFP8)
    bias, res = bf16(r, 160), bf16(r, 200, 80)
    before = mx.mx_set_batch_invariant(True)
    try:
        big = lin.run(mx, "x", bias, ref.SILU, True, res)
        for rows in (slice(0, 1), slice(90, 130), slice(199, 200)):
            assert np.array_equal(lin.run(mx, "x", bias, ref.SILU, True, res, rows=rows), big[rows])
    finally:
        mx.mx_set_batch_invariant(before)
    out, tol = ref.epilogue(lin.z, lin.dz, bias, ref.SILU, True, res)
    ops_ref.assert_within(big, out, tol, "batch-invariant")


def test_linear_epilogue_extreme_codes(g, mx):
    """bf16 activations with codes whose weights leave bf16's normal range."""
    r = rng(44)
    N, K, M = 48, 288, 5
    for elem, lo, hi in ((0, 0, 12), (1, 0, 4)):
        w = wl.e4m3_bytes(r, (1, N, K)) if elem == 0 else wl.fp4_bytes(r, (1, N, K // 2))
        codes = wl.codes(r, (N, K // 32), lo, hi)
        packed = g.pack(elem, 0, 1, N, K, w, codes)
        W = ops_ref.weights(elem, 0, 1, N, K, w, codes)[0]
        lin = Lin.__new__(Lin)
        lin.g, lin.sizes, lin.elem, lin.layout, lin.act, lin.rule = g, (M, N, K), elem, 0, BF16, 0
        lin.packed, lin.x = packed, bf16(r, M, K, scale=2.0 ** 115)
        z, dz = ref.product(ops_ref.f64(lin.x), W, False)
        res = bf16(r, M, N // 2)
        y = lin.run(mx, "x", None, ref.SILU, True, res)
        out, tol = ref.epilogue(z, dz, None, ref.SILU, True, res)
        ops_ref.assert_within(y, out, tol, "extreme codes")


# ---- together, other streams, graphs, long buffers ---------------------------------------------


class Layer:
    """A layer's second half as a program runs it: the norms around the attention
    block, the choice of experts, their products, and a shared expert beside them
    whose projection adds the experts' sum, with the next layer's norms behind it."""

    def __init__(self, g, mx, T, H=256, I=96, J=160, E=12, topk=3, key=0):
        import torch
        r = rng(60, T, key)
        self.g, self.mx, self.sizes = g, mx, (T, H, I, J, E, topk)
        self.i = block_inputs(r, T, H, True)
        self.x2, self.gate2 = None, bf16(r, 1, H, scale=0.5)
        self.w2 = bf16(r, H)
        self.logits = r.standard_normal((T, E)).astype(np.float32)
        self.logits[r.random(T) < 0.1] = -INF
        self.bias = (0.1 * r.standard_normal(E)).astype(np.float32)
        w = lambda E, N, K, elem: self._weights(r, elem, E, N, K)               # noqa: E731
        self.gu, self.dn = w(E, 2 * I, H, 1), w(E, H, I, 0)
        self.sgu, self.sdn = w(1, 2 * J, H, 0), w(1, H, J, 0)
        d = g.dev
        self.d = {k: d(v) for k, v in self.i.items()}
        self.d.update(gate2=d(self.gate2), w2=d(self.w2), logits=d(self.logits), bias=d(self.bias))
        P = T * topk
        new = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device=g.DEV)  # noqa: E731
        self.sum, self.sum2 = new(T, H, dtype=torch.float32), new(T, H, dtype=torch.float32)
        self.q, self.c = bytes_(g, T, H), bytes_(g, T, H // 32)
        qb, cb = mx.mx_act_t16_sizes(T, H)
        self.q16, self.c16 = bytes_(g, qb), bytes_(g, cb)
        self.h, self.y2 = out16(g, T, H), out16(g, T, H)
        self.ids, self.wts = new(T, topk), new(T, topk, dtype=torch.float32)
        self.off, self.rows, self.pos = new(E + 1), new(P), new(P)
        self.hid, self.ys, self.out = out16(g, P, I), out16(g, P, H), out16(g, T, H)
        self.shid, self.sout = out16(g, T, J), out16(g, T, H)
        need = max(mx.mx_grouped_workspace(1, 0, E, 2 * I, H, P, 1, 1),
                   mx.mx_grouped_workspace(0, 0, E, H, I, P, 1, 0), mx.mx_moe_sort_workspace(E, T, topk),
                   mx.mx_linear_workspace(0, 0, 2 * J, H, T, MXFP8, 1),
                   mx.mx_linear_workspace(0, 0, H, J, T, MXFP8, 0))
        self.ws = bytes_(g, need, fill=0xFF)

    def _weights(self, r, elem, E, N, K):
        w = wl.e4m3_bytes(r, (E, N, K)) if elem == 0 else wl.fp4_bytes(r, (E, N, K // 2))
        codes = wl.codes(r, (E * N, K // 32), 114, 120)
        return ops_ref.weights(elem, 0, E, N, K, w, codes), self.g.pack(elem, 0, E, N, K, w, codes)

    def run(self):
        T, H, I, J, E, topk = self.sizes
        mx, d, ws, n, P = self.mx, self.d, self.ws, self.ws.numel(), T * topk
        mx.mx_block_norm(T, H, d["x"], H, d["post"], d["gate"], 3, H, d["gids"], 1, d["res"], H, 0.9,
                         d["w"], 0.0, 1e-6, MXFP8, 0, self.sum, H, self.h, H, self.q, H, self.c, H // 32)
        mx.mx_moe_route(E, T, topk, 1, d["logits"], E, 1, d["bias"], 4, 2, 2, True, 1.5, self.ids, self.wts)
        mx.mx_moe_sort(E, T, topk, self.ids, self.off, self.rows, self.pos, ws, n)
        mx.mx_grouped_linear(1, 0, E, 2 * I, H, *self.gu[1], P, self.off, MXFP8, 0, T, None, 0, self.q, H,
                             self.c, H // 32, self.rows, 1, self.hid, I, ws, n)
        mx.mx_grouped_linear(0, 0, E, H, I, *self.dn[1], P, self.off, MXFP8, 0, P, self.hid, I, None, 0,
                             None, 0, None, 0, self.ys, H, ws, n)
        mx.mx_moe_combine(T, topk, H, P, self.ys, H, self.pos, self.wts, self.out, H)
        mx.mx_linear_epilogue(0, 0, 2 * J, H, *self.sgu[1], T, MXFP8, 0, None, 0, self.q, H, self.c, H // 32,
                              None, ref.SILU, True, None, 0, self.shid, J, ws, n)
        mx.mx_linear_epilogue(0, 0, H, J, *self.sdn[1], T, MXFP8, 0, self.shid, J, None, 0, None, 0, None,
                              0, False, self.out, H, self.sout, H, ws, n)
        mx.mx_block_norm(T, H, self.sout, H, None, d["gate2"], 1, H, None, 1, self.sum, H, 1.0, d["w2"], 0.0,
                         1e-6, T16, 1, self.sum2, H, self.y2, H, self.q16, 0, self.c16, 0)

    def outputs(self):
        return [self.sum, self.h, self.ids, self.wts, self.off, self.pos, self.out, self.shid, self.sout,
                self.sum2, self.y2, self.q16, self.c16]

    def check(self):
        """Each step against its definition on the values the step was given."""
        T, H, I, J, E, topk = self.sizes
        u, i, n = self.g.host_u16, self.i, lambda t: t.cpu().numpy()            # noqa: E731
        q, c = n(self.q), n(self.c)
        check_block((n(self.sum), u(self.h), q, c), i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.9,
                    i["w"], 0.0, 1e-6, MXFP8, 0, True)
        check_route((n(self.ids), n(self.wts)), self.logits, 1, self.bias, 4, 2, 2, topk, True, 1.5)
        off, rows, pos = ops_ref.sort(n(self.ids), E)
        assert np.array_equal(n(self.off), off) and np.array_equal(n(self.pos).reshape(T, topk), pos)
        a, m = ops_ref.activations(q, c), off[-1]
        out, tol = ops_ref.grouped(a[rows[:m]], self.gu[0], off, 1)
        ops_ref.assert_within(u(self.hid)[:m], out, tol, "gate and up")
        out, tol = ops_ref.combine(u(self.ys), pos, n(self.wts))
        ops_ref.assert_within(u(self.out), out, tol, "combine")
        z = ref.product(a, self.sgu[0][0], True)
        out, tol = ref.epilogue(*z, None, ref.SILU, True, None)
        ops_ref.assert_within(u(self.shid), out, tol, "shared gate and up")
        z = ref.product(ops_ref.activations(*oracle.quant_act(u(self.shid), 0)), self.sdn[0][0], True)
        out, tol = ref.epilogue(*z, None, ref.NONE, False, u(self.out))
        ops_ref.assert_within(u(self.sout), out, tol, "shared down and residual")
        q16, c16 = self.g.t16_unpack(n(self.q16), n(self.c16), T, H)
        check_block((n(self.sum2), u(self.y2), q16[:T, :H], c16[:T, :H // 32]), u(self.sout), None, self.gate2,
                    None, n(self.sum), 1.0, self.w2, 0.0, 1e-6, T16, 1, True)


@pytest.mark.parametrize("T", [1, 13, 64, 600])
def test_layer(g, mx, T):
    import torch
    layer = Layer(g, mx, T, key=3)
    layer.run()
    torch.cuda.synchronize()
    layer.check()


def test_layer_on_another_stream(g, mx):
    """Calls go to torch's current stream: two layers at once on two side streams."""
    import torch
    a, b, c = (Layer(g, mx, 40, key=1) for _ in range(3))
    a.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in a.outputs()]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, layer in zip(sides, (b, c)):
            with torch.cuda.stream(s):
                layer.run()
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    got = [[t.clone() for t in layer.outputs()] for layer in (b, c)]
    torch.cuda.synchronize()
    for outs in got:
        for x, y in zip(want, outs):
            assert torch.equal(x, y)


def test_layer_by_either_call_path(g, mx, monkeypatch):
    """The compiled call path and ctypes: the same launches, so the same bits; a
    stream as None, an object or a handle; a tensor of another device is refused."""
    import torch
    assert mx._mxcall is not None, "_mxcall is not built"
    a, b = Layer(g, mx, 40, key=1), Layer(g, mx, 40, key=1)
    a.run()
    side = torch.cuda.Stream()
    class Elsewhere:                                                            # noqa: E306
        device = "cuda:1"

        def get_device(self):
            return 1

        def data_ptr(self):
            return 256
    for compiled in (True, False):
        if not compiled:
            monkeypatch.setattr(mx, "_mxcall", None)
        monkeypatch.setattr(mx.lib(), "direct", {})
        b.run()
        torch.cuda.synchronize()
        for u, v in zip(a.outputs(), b.outputs()):
            assert torch.equal(u, v)
        for stream in (side, side.cuda_stream, 0, None):
            b.ids.zero_()
            b.wts.zero_()
            torch.cuda.synchronize()
            mx.mx_moe_route(12, 40, 3, 1, b.d["logits"], 12, 1, b.d["bias"], 4, 2, 2, True, 1.5, b.ids,
                            b.wts, stream)
            torch.cuda.synchronize()
            assert torch.equal(a.ids, b.ids) and torch.equal(a.wts, b.wts)
        for at in (4, 7, 14):                          # as the first, a later and the last tensor
            args = [8, 1, 2, 1, a.d["logits"], 8, 0, None, 1, 1, 1, 1, 1.0, a.ids, a.wts]
            args[at] = Elsewhere()
            with pytest.raises(ValueError, match="on cuda:1, not on the current GPU"):
                mx.mx_moe_route(*args)


def test_layer_captured(g, mx):
    """Captured and replayed, with eager work (another layer on the same workspace
    among it) and synchronizations between the replays; two graphs that share a
    workspace, replayed in turn; new inputs in the same buffers."""
    import torch
    a, b = Layer(g, mx, 70, key=1), Layer(g, mx, 70, key=2)
    b.ws = a.ws
    want = []
    for layer in (a, b):
        layer.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in layer.outputs()])
    graphs = []
    for layer in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, capture_error_mode="thread_local"):
            layer.run()
        graphs.append(gr)
    for turn in range(4):
        for k, layer in enumerate((a, b)):
            for t in layer.outputs():
                t.zero_()
            a.ws.fill_(turn)
            if turn % 2:
                (b if k == 0 else a).run()
            torch.cuda.synchronize()
            graphs[k].replay()
            torch.cuda.synchronize()
            for x, y in zip(layer.outputs(), want[k]):
                assert torch.equal(x, y)
    a.d["x"].copy_(b.d["x"])
    a.d["logits"].copy_(b.d["logits"])
    a.i["x"], a.logits = b.i["x"], b.logits
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check()


def test_far_rows(g, mx):
    """Rows whose byte offsets pass 2^32: the last rows of long buffers."""
    import torch
    M, ld, K = 70000, 32768, 64                       # 4.6 GB of bf16
    r = rng(70)
    last = np.array([0, 1, M // 2, M - 2, M - 1])
    at = torch.from_numpy(last).to(g.DEV)
    buf = torch.zeros((M, ld), dtype=torch.int16, device=g.DEV)
    i = block_inputs(r, 5, K, False, gates=1)
    buf[at, :K] = g.dev(i["x"])
    buf[at, K:2 * K] = g.dev(i["res"])
    q = bytes_(g, M, K)
    c = bytes_(g, M, K // 32)
    # x, the residual, the sum and y are columns of the one buffer
    col = lambda n: buf.data_ptr() + 2 * K * n                                  # noqa: E731
    mx.mx_block_norm(M, K, col(0), ld, g.dev(i["post"]), g.dev(i["gate"]), 1, K, None, 0, col(1), ld, 0.5,
                     g.dev(i["w"]), 0.0, 1e-6, MXFP8, 0, col(2), ld, col(3), ld, q, K, c, K // 32)
    torch.cuda.synchronize()
    h = g.host_u16(buf[at, :5 * K])
    check_block((h[:, 2 * K:3 * K], h[:, 3 * K:4 * K], q[at].cpu().numpy(), c[at].cpu().numpy()), i["x"],
                i["post"], i["gate"], None, i["res"], 0.5, i["w"], 0.0, 1e-6, MXFP8, 0, False)
    assert (h[:, 4 * K:] == 0).all()
    # routing from far rows
    E, topk = 96, 4
    x = bf16(r, 5, E)
    buf[at, :E] = g.dev(x)
    ids = torch.zeros((M, topk), dtype=torch.int32, device=g.DEV)
    w = torch.zeros((M, topk), dtype=torch.float32, device=g.DEV)
    mx.mx_moe_route(E, M, topk, 0, buf, ld, 0, None, 1, 1, 1, True, 1.0, ids, w)
    torch.cuda.synchronize()
    check_route((ids[at].cpu().numpy(), w[at].cpu().numpy()), x, 0, topk=topk)


def test_block_norm_many_rows(g, mx):
    """Far more rows than a round of the chip, in short rows: every row is written."""
    import torch
    r = rng(71)
    M, K = 300001, 32
    i = block_inputs(r, 64, K, False)
    rep = lambda a: g.dev(np.resize(a, (M,) + a.shape[1:]))                     # noqa: E731
    s, y = out16(g, M, K), out16(g, M, K)
    qb, cb = mx.mx_act_t16_sizes(M, K)
    q, c = bytes_(g, qb), bytes_(g, cb)
    mx.mx_block_norm(M, K, rep(i["x"]), K, g.dev(i["post"]), g.dev(i["gate"]), 3, K, rep(i["gids"]), 0,
                     rep(i["res"]), K, 0.5, g.dev(i["w"]), 0.0, 1e-6, T16, 0, s, K, y, K, q, 0, c, 0)
    torch.cuda.synchronize()
    hs, hy = g.host_u16(s), g.host_u16(y)
    a = (i["x"], i["post"], i["gate"], i["gids"], i["res"], 0.5, i["w"], 0.0, 1e-6, T16, 0, False)
    hq, hc = g.t16_unpack(q.cpu().numpy(), c.cpu().numpy(), M, K)
    check_block((hs[:64], hy[:64], hq[:64, :K], hc[:64, :1]), *a)
    for whole in (hs, hy, hq[:M, :K], hc[:M, :1]):
        assert np.array_equal(whole, np.resize(whole[:64], whole.shape))
