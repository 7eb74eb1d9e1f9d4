"""The operators around the linear on the GPU -- residual norm with quantized
output, expert sort, grouped products over ragged ranges, combine, low-rank
adapters -- against their plain 64-bit definitions (tests/ops_ref.py), at the
sizes, strides, masks and orders where they could go wrong, alone and run
together."""
import numpy as np
import pytest

import ops_ref as ref
import oracle
from microscaling_quantized_linear_amd import workloads as wl

pytestmark = pytest.mark.gpu

BF16, MXFP8, T16 = 0, 1, 2
NAN16 = 0x7FC1                 # a bf16 NaN that no output holds


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
    return np.random.default_rng([77, *key])


def bf16(r, *shape, scale=1.0):
    return wl.f32_to_bf16_bits(r.standard_normal(shape).astype(np.float32) * np.float32(scale))


def strided(g, a, ld):
    """A device buffer [rows, ld] with `a` in its first columns, NaN behind."""
    buf = np.full((a.shape[0], ld), NAN16, np.uint16)
    buf[:, :a.shape[1]] = a
    return g.dev(buf)


def out16(g, rows, ld):
    import torch
    return torch.full((rows, ld), NAN16, dtype=torch.int16, device=g.DEV)


def bytes_(g, *shape, fill=0xAB):
    import torch
    return torch.full(shape, fill, dtype=torch.uint8, device=g.DEV)


# ---- residual norm ----------------------------------------------------------------


def run_norm(g, mx, x, res, w, eps, act, rule, keep=True, want_sum=True, pad=0, stream=None):
    """The call's outputs on the host: (sum, y, xq, xcodes), T16 buffers unpacked
    to padded row-major; checks that nothing outside the outputs changed."""
    import torch
    M, K = x.shape
    xd, rd = strided(g, x, K + pad), strided(g, res, K + 2 * pad) if res is not None else None
    s = out16(g, M + 1, K + pad) if want_sum else None
    y = out16(g, M + 1, K + 3 * pad) if keep or act == BF16 else None
    if act == T16:
        qb, cb = mx.mx_act_t16_sizes(M, K)
        q, c, ldq, ldc = bytes_(g, qb + 16), bytes_(g, cb + 16), 0, 0
    else:
        ldq, ldc = K + 2 * pad, K // 32 + pad
        q, c = bytes_(g, M + 1, ldq), bytes_(g, M + 1, ldc)
    mx.mx_add_rms_norm(M, K, xd, K + pad, rd, K + 2 * pad if rd is not None else 0, g.dev(w), eps,
                       act, rule, s, K + pad if s is not None else 0, y,
                       K + 3 * pad if y is not None else 0, q, ldq, c, ldc, stream)
    torch.cuda.synchronize()
    hs = hy = hq = hc = None
    if s is not None:
        hs = g.host_u16(s)
        assert (hs[M:] == NAN16).all() and (hs[:, K:] == NAN16).all()
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


def check_norm(out, x, res, w, eps, act, rule):
    s, y, q, c = out
    want = ref.residual_sum(x, res)
    if s is not None:
        assert np.array_equal(s, want)
    exact = ref.rms_norm(want, w, eps)
    # the sum of squares passes at most 8 * 16 + 3 + 6 additions (half of its
    # relative error reaches the root), then a division, a root, a reciprocal
    # and two products: under 80 half steps of fp32, and one bf16 rounding
    tol = (ref.HALF_BF16 + 2.0 ** -17) * np.abs(exact)
    if y is not None:
        ref.assert_within(y, exact, tol, "norm")
    if act != BF16 and y is not None:
        oq, oc = oracle.quant_act(y, rule)
        assert np.array_equal(c, oc) and np.array_equal(q, oq)


@pytest.mark.parametrize("act", [BF16, MXFP8, T16])
@pytest.mark.parametrize("M,K,pad", [
    (1, 32, 0), (1, 7168, 0), (3, 96, 16), (16, 512, 0), (17, 544, 32), (5, 1568, 16),
    (33, 4096, 0), (2, 4128, 16), (40, 7168, 16), (2, 8192, 0), (1, 16384, 0), (2, 20000, 16),
    (1, 32768, 0), (1, 65536, 0)])
def test_norm(g, mx, M, K, pad, act):
    K = K // 32 * 32
    r = rng(1, M, K)
    x, res, w = bf16(r, M, K), bf16(r, M, K, scale=3), bf16(r, K)
    for rule, with_res in ((0, True), (1, False)):
        rr = res if with_res else None
        out = run_norm(g, mx, x, rr, w, 1e-6, act, rule, pad=pad)
        check_norm(out, x, rr, w, 1e-6, act, rule)


def test_norm_outputs_left_out(g, mx):
    """No sum, no bf16 y: the bytes stay the same."""
    r = rng(2)
    M, K = 9, 1056
    x, res, w = bf16(r, M, K), bf16(r, M, K), bf16(r, K)
    for act in (MXFP8, T16):
        full = run_norm(g, mx, x, res, w, 1e-5, act, 0)
        bare = run_norm(g, mx, x, res, w, 1e-5, act, 0, keep=False, want_sum=False)
        assert bare[0] is None and bare[1] is None
        assert np.array_equal(full[2], bare[2]) and np.array_equal(full[3], bare[3])


def test_norm_rows_do_not_depend_on_the_call(g, mx):
    """A row alone, in a small call and in a large one: the same bits."""
    r = rng(3)
    for K in (512, 1568, 7168):
        M = 700
        x, res, w = bf16(r, M, K), bf16(r, M, K, scale=2), bf16(r, K)
        big = run_norm(g, mx, x, res, w, 1e-6, T16, 0)
        for m0, m1 in ((0, 1), (5, 22), (698, 700)):
            part = run_norm(g, mx, x[m0:m1], res[m0:m1], w, 1e-6, T16, 0)
            for a, b in zip(big, part):
                assert np.array_equal(a[m0:m1], b)


def test_norm_ranges(g, mx):
    """Zero rows (also with eps 0.5), tiny and large values, saturating blocks."""
    r = rng(4)
    M, K = 6, 128
    x = bf16(r, M, K)
    x[0] = 0
    x[1] = bf16(r, K, scale=1e-18)
    x[2] = bf16(r, K, scale=1e17)
    x[3] = 0x8000                                   # -0
    w = bf16(r, K, scale=4)
    w[5], w[6] = 0, 0x8000
    for act in (MXFP8, T16):
        for rule in (0, 1):
            check_norm(run_norm(g, mx, x, None, w, 0.5, act, rule), x, None, w, 0.5, act, rule)
            check_norm(run_norm(g, mx, x, None, w, 1e-12, act, rule), x, None, w, 1e-12, act, rule)


@pytest.mark.parametrize("M,K", [(1, 64), (19, 7168), (130, 1568)])
def test_norm_in_place(g, mx, M, K):
    """sum on the residual, y on x: the separate call's values."""
    import torch
    r = rng(5, M, K)
    x, res, w = bf16(r, M, K), bf16(r, M, K), bf16(r, K)
    s, y, _, _ = run_norm(g, mx, x, res, w, 1e-6, BF16, 0)
    xd, rd, wd = g.dev(x), g.dev(res), g.dev(w)
    mx.mx_add_rms_norm(M, K, xd, K, rd, K, wd, 1e-6, BF16, 0, rd, K, xd, K, None, 0, None, 0)
    torch.cuda.synchronize()
    assert np.array_equal(g.host_u16(rd), s) and np.array_equal(g.host_u16(xd), y)
    xd, rd = g.dev(x), g.dev(res)
    mx.mx_add_rms_norm(M, K, xd, K, rd, K, wd, 1e-6, BF16, 0, xd, K, rd, K, None, 0, None, 0)
    torch.cuda.synchronize()
    assert np.array_equal(g.host_u16(xd), s) and np.array_equal(g.host_u16(rd), y)


# ---- sort ---------------------------------------------------------------------------


def run_sort(g, mx, ids, E, stream=None):
    import torch
    T, topk = ids.shape
    P = T * topk
    off = torch.full((E + 2,), -7, dtype=torch.int32, device=g.DEV)
    rows = torch.full((P + 1,), -7, dtype=torch.int32, device=g.DEV)
    pos = torch.full((P + 1,), -7, dtype=torch.int32, device=g.DEV)
    need = mx.mx_moe_sort_workspace(E, T, topk)
    ws = bytes_(g, max(need, 16), fill=0x5A)
    mx.mx_moe_sort(E, T, topk, g.dev(ids), off, rows, pos, ws if need else None, need, stream)
    torch.cuda.synchronize()
    assert int(off[-1]) == -7 and int(rows[-1]) == -7 and int(pos[-1]) == -7
    return (off[:-1].cpu().numpy(), rows[:-1].cpu().numpy(),
            pos[:-1].cpu().numpy().reshape(T, topk))


def routed(r, E, T, topk, drop=0.0, skew=0.0):
    logits = r.standard_normal((T, E)) + skew * r.standard_normal(E)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :topk].astype(np.int32)
    ids[r.random(T) < drop] = -1
    return ids


@pytest.mark.parametrize("E,T,topk,drop,skew", [
    (1, 1, 1, 0, 0), (2, 1, 2, 0, 0), (8, 5, 2, 0, 0), (32, 16, 8, 0, 0.5), (64, 63, 3, 0.3, 2),
    (256, 33, 8, 0, 0), (256, 256, 8, 0.1, 1), (256, 257, 8, 0.1, 1), (7, 2049, 1, 0, 3),
    (128, 4096, 8, 0.05, 1), (1000, 700, 8, 0, 1), (1024, 1500, 16, 0.2, 0), (3, 60000, 2, 0, 1),
    (511, 9000, 6, 0, 0), (512, 9000, 6, 0, 0), (32, 100003, 8, 0.5, 4)])
def test_sort(g, mx, E, T, topk, drop, skew):
    ids = routed(rng(10, E, T), E, T, topk, drop, skew)
    for got, want in zip(run_sort(g, mx, ids, E), ref.sort(ids, E)):
        assert np.array_equal(got, want)


def test_sort_odd_ids(g, mx):
    """No pair with an expert; one expert only; an id twice in a token; ids far
    outside the range."""
    r = rng(11)
    for T in (3, 700, 5000):
        E, topk = 12, 4
        for ids in (np.full((T, topk), -1), np.full((T, topk), 11), np.full((T, topk), 12),
                    r.integers(-2, E + 2, (T, topk)),
                    r.choice([-2 ** 31, 2 ** 31 - 1, 0, 5], (T, topk))):
            ids = ids.astype(np.int32)
            for got, want in zip(run_sort(g, mx, ids, E), ref.sort(ids, E)):
                assert np.array_equal(got, want)


# ---- grouped products ------------------------------------------------------------------


def weight(g, r, elem, layout, E, N, K, lo=118, hi=132):
    w = wl.e4m3_bytes(r, (E, N, K)) if elem == 0 else wl.fp4_bytes(r, (E, N, K // 2))
    codes = wl.codes(r, (E * N // (32 if layout else 1), K // 32), lo, hi)
    return w, codes, g.pack(elem, layout, E, N, K, w, codes)


def run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, x=None, given=None, rows=None,
                rule=0, epi=0, pad=0, t16=None, stream=None):
    import torch
    width = N // 2 if epi else N
    ldy = (width + 7) // 8 * 8 + pad
    y = out16(g, M + 1, ldy)
    act = T16 if t16 is not None else MXFP8
    need = mx.mx_grouped_workspace(elem, layout, E, N, K, M, act, given is not None)
    ws = bytes_(g, max(need, 16), fill=0x7F)          # NaN bytes: unstaged ones must not be read
    off, rd = g.dev(np.asarray(offsets, np.int32)), g.dev(rows) if rows is not None else None
    kw = dict(xd=None, ldx=0, q=None, ldq=0, c=None, ldc=0, xrows=0)
    if t16 is not None:
        kw.update(q=t16[0], c=t16[1])
    elif given is not None:
        q, c = given
        ldq = (K + 15) // 16 * 16 + pad
        buf = np.full((q.shape[0], ldq), 0x7F, np.uint8)
        buf[:, :K] = q
        cb = np.full((c.shape[0], K // 32 + 3), 0xFF, np.uint8)
        cb[:, :K // 32] = c
        kw.update(q=g.dev(buf), ldq=ldq, c=g.dev(cb), ldc=K // 32 + 3, xrows=q.shape[0])
    else:
        kw.update(xd=strided(g, x, K + pad), ldx=K + pad, xrows=x.shape[0])
    mx.mx_grouped_linear(elem, layout, E, N, K, *packed, M, off, act, rule, kw["xrows"], kw["xd"],
                         kw["ldx"], kw["q"], kw["ldq"], kw["c"], kw["ldc"], rd, epi, y, ldy,
                         ws if need else None, need, stream)
    torch.cuda.synchronize()
    h = g.host_u16(y)
    lo = max(0, int(offsets[0]))
    hi = max(lo, min(M, int(offsets[-1])))
    assert (h[hi:] == NAN16).all() and (h[:lo] == NAN16).all() and (h[:, width:] == NAN16).all()
    return h[:M, :width]


def check_grouped(y, a, w, offsets, epi, what=""):
    out, tol = ref.grouped(a, w, offsets, epi)
    lo, hi = int(offsets[0]), int(offsets[-1])
    ref.assert_within(y[lo:hi], out[lo:hi], tol[lo:hi], what)
    # The linear's own bar on enough plain products.  It does not carry over to the
    # SiLU product: where a result's L2 norm sits in few values it asks for one bf16
    # step (2^-7 of the value) of each, but a gate is off by up to 7 * 2^-13 of its
    # sum of magnitudes, so a gate of a tenth of that sum by 7 * 10 * 2^-13 = 2^-6.9
    # of itself, and with it the product.
    if not epi and (hi - lo) * y.shape[1] >= 4096:
        import mxgpu
        mxgpu.assert_close(np.ascontiguousarray(y[lo:hi]), out[lo:hi], what)


def split(r, M, E, kind):
    """Row counts of E experts that sum to M."""
    if kind == "one":                                # a single expert takes them all
        n = np.zeros(E, int)
        n[E // 2] = M
    elif kind == "skew":
        n = r.multinomial(M, r.dirichlet(np.full(E, 0.3)))
    else:
        n = r.multinomial(M, np.full(E, 1.0 / E))
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


FORMS = [(0, 0), (0, 1), (1, 0)]                      # (elem, layout)
SHAPES = [  # E, N, K, M, split
    (1, 32, 32, 1, "even"), (2, 64, 96, 3, "even"), (4, 32, 128, 5, "one"),
    (8, 256, 512, 16, "even"), (5, 96, 1568, 7, "skew"), (3, 64, 160, 100, "skew"),
    (6, 288, 544, 200, "even"), (4, 512, 1024, 300, "skew"), (2, 224, 2048, 129, "one"),
    (16, 128, 640, 33, "skew"), (2, 544, 416, 700, "skew"), (3, 1024, 768, 1500, "even"),
    # enough weight panels for the tiled form at few rows, and for its 256-row tiles
    (130, 48 + 16, 544, 1300, "skew"), (64, 544, 1056, 640, "even"), (140, 32, 2080, 2000, "one"),
    (512, 32, 96, 4000, "skew"), (300, 288, 160, 2500, "skew"), (520, 64, 1184, 9000, "even"),
    (130, 288, 160, 17000, "even")]


@pytest.mark.parametrize("elem,layout", FORMS)
@pytest.mark.parametrize("E,N,K,M,kind", SHAPES)
def test_grouped(g, mx, E, N, K, M, kind, elem, layout):
    r = rng(20, E, N, K, M, elem, layout)
    w, codes, packed = weight(g, r, elem, layout, E, N, K)
    W = ref.weights(elem, layout, E, N, K, w, codes)
    offsets = split(r, M, E, kind)
    x = wl.activations(r, (M, K), 0.01)
    for rule, epi in ((0, 0), (1, 1)):
        q, c = oracle.quant_act(x, rule)
        a = ref.activations(q, c)
        y = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, x=x, rule=rule, epi=epi)
        check_grouped(y, a, W, offsets, epi, f"rule {rule} epi {epi}")
        # the same bits from rows quantized ahead, row-major and T16
        y2 = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, given=(q, c), epi=epi,
                         pad=16)
        y3 = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M,
                         t16=g.quant_t16(x, rule), epi=epi)
        assert np.array_equal(y, y2) and np.array_equal(y, y3)


@pytest.mark.parametrize("elem,layout", FORMS)
def test_grouped_by_index(g, mx, elem, layout):
    """Rows gathered by index, some without a source; ranges that end before M."""
    E, N, K, T, M = 6, 160, 736, 23, 90
    r = rng(21, elem, layout)
    w, codes, packed = weight(g, r, elem, layout, E, N, K)
    W = ref.weights(elem, layout, E, N, K, w, codes)
    offsets = split(r, 77, E, "skew")
    rows = r.integers(0, T, M).astype(np.int32)
    rows[[3, 20, 50]] = (-1, T, 2 ** 31 - 1)
    x = wl.activations(r, (T, K), 0.01)
    q, c = oracle.quant_act(x, 0)
    a = np.where(((rows >= 0) & (rows < T))[:, None],
                 ref.activations(q, c)[np.clip(rows, 0, T - 1)], 0.0)
    y = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, x=x, rows=rows, pad=24)
    check_grouped(y, a, W, offsets, 0)
    y2 = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, given=(q, c), rows=rows)
    assert np.array_equal(y[:77], y2[:77])


def test_grouped_offsets(g, mx):
    """No rows at all; ranges that start behind row 0; offsets outside 0 .. M are
    cut off (the neighbours of a range keep their rows)."""
    E, N, K, M = 4, 64, 256, 40
    r = rng(22)
    w, codes, packed = weight(g, r, 0, 0, E, N, K)
    W = ref.weights(0, 0, E, N, K, w, codes)
    x = wl.activations(r, (M, K))
    a = ref.activations(*oracle.quant_act(x, 0))
    for offsets in ([0, 0, 0, 0, 0], [5, 9, 9, 30, 31], [40, 40, 40, 40, 40], [0, 0, 0, 0, 40]):
        y = run_grouped(g, mx, 0, 0, E, N, K, packed, offsets, M, x=x)
        check_grouped(y, a, W, offsets, 0)
    y = run_grouped(g, mx, 0, 0, E, N, K, packed, [-5, 10, 20, 30, 1000], M, x=x)
    check_grouped(y, a, W, [0, 10, 20, 30, 40], 0)


@pytest.mark.parametrize("elem,layout", FORMS)
def test_grouped_extreme_codes(g, mx, elem, layout):
    """E8M0 codes at both ends of what keeps the products in fp32's range."""
    E, N, K, M = 2, 64, 192, 20
    r = rng(23, elem, layout)
    x = wl.activations(r, (M, K))
    a = ref.activations(*oracle.quant_act(x, 0))
    offsets = split(r, M, E, "even")
    for lo, hi in ((10, 40), (200, 230)):
        w, codes, packed = weight(g, r, elem, layout, E, N, K, lo, hi)
        W = ref.weights(elem, layout, E, N, K, w, codes)
        y = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, x=x)
        check_grouped(y, a, W, offsets, 0)


def test_grouped_zero_blocks_and_neighbours(g, mx):
    """Rows of one expert do not touch another's: huge rows beside zero rows."""
    E, N, K, M = 3, 96, 320, 50
    r = rng(24)
    w, codes, packed = weight(g, r, 1, 0, E, N, K)
    W = ref.weights(1, 0, E, N, K, w, codes)
    x = wl.activations(r, (M, K))
    x[17:33] = bf16(r, 16, K, scale=1e30)
    x[33:40] = 0
    offsets = [0, 17, 33, 50]
    a = ref.activations(*oracle.quant_act(x, 0))
    y = run_grouped(g, mx, 1, 0, E, N, K, packed, offsets, M, x=x)
    check_grouped(y, a, W, offsets, 0)
    assert (y[33:40] & 0x7FFF == 0).all()


def test_grouped_many_experts(g, mx):
    E, N, K, M = 300, 32, 64, 500
    r = rng(25)
    for elem in (0, 1):
        w, codes, packed = weight(g, r, elem, 0, E, N, K)
        W = ref.weights(elem, 0, E, N, K, w, codes)
        x = wl.activations(r, (M, K))
        a = ref.activations(*oracle.quant_act(x, 0))
        for kind in ("even", "skew"):
            offsets = split(r, M, E, kind)
            y = run_grouped(g, mx, elem, 0, E, N, K, packed, offsets, M, x=x)
            check_grouped(y, a, W, offsets, 0)


def test_grouped_beyond_the_tile_table(g, mx):
    """More experts than the tiled form counts (1024): the streaming form serves
    them, also with many rows."""
    E, N, K, M = 1100, 32, 64, 9000
    r = rng(26)
    w, codes, packed = weight(g, r, 1, 0, E, N, K)
    W = ref.weights(1, 0, E, N, K, w, codes)
    x = wl.activations(r, (M, K))
    a = ref.activations(*oracle.quant_act(x, 0))
    offsets = split(r, M, E, "skew")
    y = run_grouped(g, mx, 1, 0, E, N, K, packed, offsets, M, x=x)
    check_grouped(y, a, W, offsets, 0)


@pytest.mark.parametrize("E,N,K,M", [
    (512, 96, 544, 1500), (270, 160, 288, 700), (1030, 96, 96, 12000), (1030, 96, 160, 25000)])
def test_grouped_panels_cut_short(g, mx, E, N, K, M):
    """Many experts: the streaming form's panels of four weight tiles, the last
    of an expert with fewer, at each of its batch sizes."""
    r = rng(27, E, M)
    w, codes, packed = weight(g, r, 1, 0, E, N, K)
    W = ref.weights(1, 0, E, N, K, w, codes)
    x = wl.activations(r, (M, K))
    a = ref.activations(*oracle.quant_act(x, 0))
    offsets = split(r, M, E, "skew")
    for epi in (0, 1):
        y = run_grouped(g, mx, 1, 0, E, N, K, packed, offsets, M, x=x, epi=epi)
        check_grouped(y, a, W, offsets, epi)


def test_grouped_descending_offsets_stay_inside(g, mx):
    """Offsets that descend: which rows are written is unspecified, but only rows
    of y are, and the call ends."""
    import torch
    r = rng(27)
    for E, N, K, M in ((4, 64, 256, 40), (200, 64, 256, 3000)):
        w, codes, packed = weight(g, r, 0, 0, E, N, K)
        x = wl.activations(r, (M, K))
        offsets = r.integers(-50, M + 50, E + 1).astype(np.int32)
        y = out16(g, M + 4, N)
        need = mx.mx_grouped_workspace(0, 0, E, N, K, M, 1, 0)
        ws = bytes_(g, need)
        mx.mx_grouped_linear(0, 0, E, N, K, *packed, M, g.dev(offsets), MXFP8, 0, M, g.dev(x), K,
                             None, 0, None, 0, None, 0, y, N, ws, need)
        torch.cuda.synchronize()
        assert (g.host_u16(y)[M:] == NAN16).all()


def test_batch_invariant_mode(g, mx):
    """With the mode on, a row's grouped product and its adapter's do not depend
    on the rows beside it: alone, in a small call and in a large one."""
    r = rng(28)
    E, N, K, M = 3, 288, 1056, 900
    w, codes, packed = weight(g, r, 1, 0, E, N, K)
    x = wl.activations(r, (M, K), 0.01)
    offsets = np.array([0, 300, 310, 900], np.int32)
    la, lb, ls, lx, ids, base = lora_inputs(r, 4, 24, N, K, M, "mixed")
    before = mx.mx_set_batch_invariant(True)
    try:
        big = run_grouped(g, mx, 1, 0, E, N, K, packed, offsets, M, x=x)
        blora = run_lora(g, mx, la, lb, ls, lx, ids, base)
        for m0, m1 in ((0, 1), (290, 330), (880, 900)):
            off = np.clip(offsets - m0, 0, m1 - m0)
            part = run_grouped(g, mx, 1, 0, E, N, K, packed, off, m1 - m0, x=x[m0:m1])
            assert np.array_equal(part, big[m0:m1])
            part = run_lora(g, mx, la, lb, ls, lx[m0:m1], ids[m0:m1], base[m0:m1])
            assert np.array_equal(part, blora[m0:m1])
    finally:
        mx.mx_set_batch_invariant(before)
    W = ref.weights(1, 0, E, N, K, w, codes)
    check_grouped(big, ref.activations(*oracle.quant_act(x, 0)), W, offsets, 0)


# ---- combine ----------------------------------------------------------------------------


@pytest.mark.parametrize("T,topk,N,M,pad", [
    (1, 1, 8, 1, 0), (3, 2, 24, 7, 8), (16, 8, 7168, 128, 0), (5, 5, 2048, 11, 16),
    (7, 9, 2056, 63, 8), (300, 3, 264, 100, 0)])
def test_combine(g, mx, T, topk, N, M, pad):
    import torch
    r = rng(30, T, N)
    ys = bf16(r, M, N)
    pos = r.integers(-1, M, (T, topk)).astype(np.int32)
    far = r.random((T, topk)) < 0.1
    pos[far] = r.choice([M, 2 ** 31 - 1, -2 ** 31], far.sum())
    pos[T // 2] = -1                                  # a token without places
    gone = (pos < 0) | (pos >= M)
    wts = r.standard_normal((T, topk)).astype(np.float32)
    wts[gone] = np.nan                                # not read
    ys[np.setdiff1d(np.arange(M), pos)] = NAN16
    y = out16(g, T + 1, N + pad)
    mx.mx_moe_combine(T, topk, N, M, strided(g, ys, N + 2 * pad), N + 2 * pad, g.dev(pos),
                      g.dev(wts), y, N + pad)
    torch.cuda.synchronize()
    h = g.host_u16(y)
    assert (h[T:] == NAN16).all() and (h[:, N:] == NAN16).all()
    out, tol = ref.combine(ys, pos, np.where(gone, 0, wts))
    ref.assert_within(h[:T, :N], out, tol, "combine")
    assert (h[T // 2, :N] == 0).all()


# ---- adapters -----------------------------------------------------------------------------


def run_lora(g, mx, a, b, scales, x, ids, base, pad=0, inplace=False, stream=None):
    import torch
    (L, R, K), N, M = a.shape, b.shape[1], x.shape[0]
    need = mx.mx_lora_workspace(L, R, N, K, M)
    ws = bytes_(g, need, fill=0xFF)                   # NaN: what is not written must not be read
    xd = strided(g, x, K + pad)
    bd = strided(g, base, N + pad)
    y = bd if inplace else out16(g, M + 1, N + 2 * pad)
    ldy = N + pad if inplace else N + 2 * pad
    mx.mx_lora_add(L, R, N, K, g.dev(a), g.dev(b), None if scales is None else g.dev(scales), M, xd,
                   K + pad, g.dev(ids), bd, N + pad, y, ldy, ws, need, stream)
    torch.cuda.synchronize()
    h = g.host_u16(y)
    assert (h[M:] == NAN16).all() and (h[:, N:] == NAN16).all()
    return h[:M, :N]


def lora_inputs(r, L, R, N, K, M, kind):
    a, b = bf16(r, L, R, K, scale=K ** -0.5), bf16(r, L, N, R, scale=R ** -0.5)
    if kind == "each":
        ids = r.permutation(np.arange(M) % L)
    elif kind == "runs":
        ids = np.sort(r.integers(0, L, M))
    elif kind == "none":
        ids = np.full(M, -1)
    else:
        ids = r.integers(-1, L + 1, M)                # -1 and L: no adapter
    return a, b, (0.5 + r.random(L)).astype(np.float32), bf16(r, M, K), ids.astype(np.int32), \
        bf16(r, M, N)


@pytest.mark.parametrize("L,R,N,K,M,kind,pad", [
    (1, 8, 16, 32, 1, "runs", 0), (4, 16, 64, 64, 5, "mixed", 8), (32, 16, 512, 512, 16, "each", 0),
    (3, 24, 80, 96, 17, "mixed", 16), (8, 32, 272, 1568, 40, "each", 0),
    (2, 40, 128, 7168, 3, "runs", 0), (5, 64, 336, 2080, 33, "mixed", 8),
    (20, 128, 96, 256, 20, "each", 0), (3, 256, 64, 160, 18, "mixed", 8),
    (4, 8, 1024, 4096, 100, "none", 0), (6, 16, 304, 288, 511, "mixed", 0),
    (6, 16, 304, 288, 512, "runs", 8), (7, 64, 512, 1088, 700, "mixed", 0),
    (64, 8, 64, 96, 600, "each", 0), (2, 256, 272, 64, 515, "runs", 0),
    (3, 72, 48, 2176, 1000, "mixed", 16)])
def test_lora(g, mx, L, R, N, K, M, kind, pad):
    a, b, s, x, ids, base = lora_inputs(rng(40, L, R, M), L, R, N, K, M, kind)
    out, tol = ref.lora(x, a, b, s, ids, base)
    y = run_lora(g, mx, a, b, s, x, ids, base, pad)
    ref.assert_within(y, out, tol, "lora")
    none = (ids < 0) | (ids >= L)
    assert np.array_equal(y[none], base[none])
    assert np.array_equal(run_lora(g, mx, a, b, s, x, ids, base, pad, inplace=True), y)
    out, tol = ref.lora(x, a, b, None, ids, base)
    ref.assert_within(run_lora(g, mx, a, b, None, x, ids, base, pad), out, tol, "lora, no scales")


def test_lora_rows_without_adapter_are_not_read(g, mx):
    """NaN rows of x without an adapter leave the others, and their own base, alone."""
    for M in (20, 600):
        a, b, s, x, ids, base = lora_inputs(rng(41, M), 5, 16, 96, 160, M, "mixed")
        none = (ids < 0) | (ids >= 5)
        out, tol = ref.lora(x, a, b, s, ids, base)
        x[none] = NAN16
        y = run_lora(g, mx, a, b, s, x, ids, base)
        ref.assert_within(y, out, tol, "lora")


@pytest.mark.parametrize("R", [8, 24, 40, 72])
@pytest.mark.parametrize("M", [20, 600])
def test_lora_infinite_inputs(g, mx, M, R):
    """With positive A and B an infinite x makes its row infinite (not NaN), and
    leaves the other rows alone."""
    a, b, s, x, ids, base = lora_inputs(rng(42, M, R), 5, R, 96, 160, M, "each")
    a, b = a & 0x7FFF | 0x0080, b & 0x7FFF | 0x0080       # positive, none zero
    out, tol = ref.lora(x, a, b, s, ids, base)
    up, down = np.arange(1, M, 7), np.arange(3, M, 7)
    x[up, up % 160], x[down, down % 160] = 0x7F80, 0xFF80
    rest = np.setdiff1d(np.arange(M), np.concatenate([up, down]))
    y = run_lora(g, mx, a, b, s, x, ids, base)
    assert (y[up] == 0x7F80).all() and (y[down] == 0xFF80).all()
    ref.assert_within(y[rest], out[rest], tol[rest], "lora")


# ---- together, other streams, graphs, long buffers ---------------------------------------------


def to_host(t):
    return t.cpu().numpy()


class Layer:
    """A quantized layer's tail as a program runs it: norm -> shared projection
    with adapters, and norm -> sort -> gate/up -> down -> combine."""

    def __init__(self, g, mx, T, H=256, I=96, N=320, E=6, topk=2, L=3, R=16, key=0):
        import torch
        r = rng(50, T, key)
        self.g, self.mx = g, mx
        self.sizes = (T, H, I, N, E, topk, L, R)
        self.x, self.res, self.w = bf16(r, T, H), bf16(r, T, H), bf16(r, H)
        self.ids = routed(r, E, T, topk, 0.1)
        self.wts = r.random((T, topk)).astype(np.float32)
        self.p_w, self.p_c, self.p = weight(g, r, 0, 1, 1, N, H, 118, 124)
        self.g_w, self.g_c, self.gu = weight(g, r, 1, 0, E, 2 * I, H, 118, 124)
        self.d_w, self.d_c, self.dn = weight(g, r, 0, 0, E, H, I, 114, 120)
        self.a, self.b, self.s, _, self.aid, _ = lora_inputs(r, L, R, N, H, T, "mixed")
        d = g.dev
        self.d = {k: d(getattr(self, k))
                  for k in ("x", "res", "w", "ids", "wts", "a", "b", "s", "aid")}
        P = T * topk
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=g.DEV)  # noqa: E731
        self.sum, self.h = out16(g, T, H), out16(g, T, H)
        self.q, self.c = bytes_(g, T, H), bytes_(g, T, H // 32)
        qb, cb = mx.mx_act_t16_sizes(T, H)
        self.q16, self.c16 = bytes_(g, qb), bytes_(g, cb)
        self.y = out16(g, T, N)
        self.off, self.rows, self.pos = i32(E + 1), i32(P), i32(P)
        self.hid, self.ys, self.out = out16(g, P, I), out16(g, P, H), out16(g, T, H)
        need = max(mx.mx_grouped_workspace(1, 0, E, 2 * I, H, P, 1, 1),
                   mx.mx_grouped_workspace(0, 0, E, H, I, P, 1, 0),
                   mx.mx_lora_workspace(L, R, N, H, T), mx.mx_moe_sort_workspace(E, T, topk))
        self.ws = bytes_(g, need, fill=0xFF)

    def run(self):
        T, H, I, N, E, topk, L, R = self.sizes
        mx, d, ws, n = self.mx, self.d, self.ws, self.ws.numel()
        mx.mx_add_rms_norm(T, H, d["x"], H, d["res"], H, d["w"], 1e-6, T16, 0, self.sum, H, None, 0,
                           self.q16, 0, self.c16, 0)
        mx.mx_linear(0, 1, N, H, *self.p, T, T16, 0, None, 0, self.q16, 0, self.c16, 0, None,
                     self.y, N, None, 0)
        mx.mx_add_rms_norm(T, H, d["x"], H, d["res"], H, d["w"], 1e-6, MXFP8, 0, None, 0, self.h, H,
                           self.q, H, self.c, H // 32)
        mx.mx_lora_add(L, R, N, H, d["a"], d["b"], d["s"], T, self.h, H, d["aid"], self.y, N,
                       self.y, N, ws, n)
        mx.mx_moe_sort(E, T, topk, d["ids"], self.off, self.rows, self.pos, ws, n)
        P = T * topk
        mx.mx_grouped_linear(1, 0, E, 2 * I, H, *self.gu, P, self.off, MXFP8, 0, T, None, 0, self.q,
                             H, self.c, H // 32, self.rows, 1, self.hid, I, ws, n)
        mx.mx_grouped_linear(0, 0, E, H, I, *self.dn, P, self.off, MXFP8, 0, P, self.hid, I, None,
                             0, None, 0, None, 0, self.ys, H, ws, n)
        mx.mx_moe_combine(T, topk, H, P, self.ys, H, self.pos, d["wts"], self.out, H)

    def outputs(self):
        return [self.sum, self.h, self.y, self.off, self.pos, self.out]

    def check(self):
        """Each step against its definition on the values the step was given."""
        T, H, I, N, E, topk, L, R = self.sizes
        u = self.g.host_u16
        s, h = u(self.sum), u(self.h)
        check_norm((s, h, None, None), self.x, self.res, self.w, 1e-6, BF16, 0)
        q, c = oracle.quant_act(h, 0)
        assert np.array_equal(to_host(self.q), q) and np.array_equal(to_host(self.c), c)
        a = ref.activations(q, c)
        base = ref.grouped(a, ref.weights(0, 1, 1, N, H, self.p_w, self.p_c), [0, T], 0)
        # the projection is rounded to bf16 before the adapters: its bound carries over
        bits = wl.f32_to_bf16_bits(base[0].astype(np.float32))
        out, tol = ref.lora(h, self.a, self.b, self.s, self.aid, bits)
        live = (self.aid >= 0) & (self.aid < L)
        ref.assert_within(u(self.y), out, tol + 2.5 * base[1], "projection and adapters")
        offsets, rows, pos = ref.sort(self.ids, E)
        assert np.array_equal(to_host(self.off), offsets)
        assert np.array_equal(to_host(self.rows), rows)
        assert np.array_equal(to_host(self.pos).reshape(T, topk), pos)
        n = offsets[-1]
        hid, ys = u(self.hid), u(self.ys)
        out, tol = ref.grouped(a[rows[:n]], ref.weights(1, 0, E, 2 * I, H, self.g_w, self.g_c),
                               offsets, 1)
        ref.assert_within(hid[:n], out, tol, "gate and up")
        a2 = ref.activations(*oracle.quant_act(hid[:n], 0))
        out, tol = ref.grouped(a2, ref.weights(0, 0, E, H, I, self.d_w, self.d_c), offsets, 0)
        ref.assert_within(ys[:n], out, tol, "down")
        out, tol = ref.combine(ys, pos, self.wts)
        ref.assert_within(u(self.out), out, tol, "combine")
        assert live.any()


@pytest.mark.parametrize("T", [1, 13, 64, 600])
def test_layer(g, mx, T):
    import torch
    layer = Layer(g, mx, T, key=3)
    if T == 1:                                        # the one token has an expert and an adapter
        layer.ids[:] = [[4, 1]]
        layer.aid[:] = 2
        layer.d["ids"], layer.d["aid"] = g.dev(layer.ids), g.dev(layer.aid)
    layer.run()
    torch.cuda.synchronize()
    layer.check()


def test_layer_on_another_stream(g, mx):
    """Calls go to torch's current stream: on a side stream, ordered by events
    with work on the default stream only."""
    import torch
    a, b = Layer(g, mx, 40, key=1), Layer(g, mx, 40, key=1)
    a.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in a.outputs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            b.run()
    torch.cuda.current_stream().wait_stream(side)
    got = [t.clone() for t in b.outputs()]
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_layer_captured(g, mx):
    """Captured and replayed, with eager work (another layer on the same
    workspace among it) and synchronizations between the replays; two graphs
    that share a workspace, replayed in turn; new inputs in the same buffers."""
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
    a.d["ids"].copy_(b.d["ids"])
    a.x, a.ids = b.x, b.ids
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check()


def test_far_rows(g, mx):
    """Rows whose byte offsets pass 2^32: the last rows of long buffers."""
    import torch
    M, ld, K = 70000, 32768, 64                       # 4.6 GB of bf16
    r = rng(60)
    last = np.array([0, 1, M // 2, M - 2, M - 1])
    buf = torch.zeros((M, ld), dtype=torch.int16, device=g.DEV)
    x = bf16(r, 5, K)
    at = torch.from_numpy(last).to(g.DEV)
    buf[at, :K] = g.dev(x)
    w = bf16(r, K)
    y = out16(g, M, K)
    mx.mx_add_rms_norm(M, K, buf, ld, None, 0, g.dev(w), 1e-6, BF16, 0, None, 0, y, K, None, 0,
                       None, 0)
    torch.cuda.synchronize()
    check_norm((None, g.host_u16(y[at]), None, None), x, None, w, 1e-6, BF16, 0)
    # combine from far rows, and to them
    pos = last[::-1].astype(np.int32).reshape(1, 5).copy()
    wts = r.random((1, 5)).astype(np.float32)
    out = out16(g, 1, K)
    mx.mx_moe_combine(1, 5, K, M, buf, ld, g.dev(pos), g.dev(wts), out, K)
    torch.cuda.synchronize()
    full, tol = ref.combine(x, np.array([[4, 3, 2, 1, 0]], np.int32), wts)
    ref.assert_within(g.host_u16(out), full, tol, "far combine")
    # adapters: x and y far apart
    L, R, N = 2, 8, 32
    a, b, s, _, _, _ = lora_inputs(r, L, R, N, K, 4, "each")
    ids = np.full(M, -1, np.int32)
    ids[last] = [0, 1, 0, 1, 1]
    base = torch.zeros((M, N), dtype=torch.int16, device=g.DEV)
    need = mx.mx_lora_workspace(L, R, N, K, M)
    ws = bytes_(g, need, fill=0xFF)
    mx.mx_lora_add(L, R, N, K, g.dev(a), g.dev(b), g.dev(s), M, buf, ld, g.dev(ids), base, N, base,
                   N, ws, need)
    torch.cuda.synchronize()
    full, tol = ref.lora(x, a, b, s, ids[last], np.zeros((5, N), np.uint16))
    ref.assert_within(g.host_u16(base[at]), full, tol, "far lora")
    assert int(torch.count_nonzero(base)) <= 5 * N
    # grouped: gathered from far rows
    E = 2
    wt, codes, packed = weight(g, r, 0, 0, E, N, K)
    y = out16(g, 5, N)
    need = mx.mx_grouped_workspace(0, 0, E, N, K, 5, 1, 0)
    ws = bytes_(g, need)
    mx.mx_grouped_linear(0, 0, E, N, K, *packed, 5, g.dev(np.array([0, 2, 5], np.int32)), MXFP8, 0,
                         M, buf, ld, None, 0, None, 0, g.dev(last.astype(np.int32)), 0, y, N, ws,
                         need)
    torch.cuda.synchronize()
    act = ref.activations(*oracle.quant_act(x, 0))
    check_grouped(g.host_u16(y), act, ref.weights(0, 0, E, N, K, wt, codes), [0, 2, 5], 0)
