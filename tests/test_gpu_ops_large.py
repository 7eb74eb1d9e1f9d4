"""The operators around the linear at the largest counts that they take (four
million rows or pairs) and with weights whose bytes pass 2^32.  Inputs repeat
with a period, so the definitions are computed for one period only."""
import numpy as np
import pytest

import ops_ref as ref
import oracle
from microscaling_quantized_linear_amd import workloads as wl
from test_gpu_ops import (BF16, MXFP8, NAN16, T16, bf16, bytes_, check_grouped,  # noqa: F401
                          check_norm, g, lora_inputs, mx, out16, rng, weight)

pytestmark = pytest.mark.gpu

MOST, PERIOD = 4000000, 1000


@pytest.fixture(scope="module", autouse=True)
def give_back():
    """The buffers of some gigabytes go back to the device behind these tests."""
    yield
    import torch
    torch.cuda.empty_cache()


def same_as_first(t):
    """Every period of rows holds the first one's bits."""
    import torch
    v = t.view(MOST // PERIOD, PERIOD, -1)
    return torch.equal(v, v[:1].expand_as(v))


def test_norm_of_the_most_rows(g, mx):
    import torch
    K = 32
    r = rng(110)
    x, w = bf16(r, PERIOD, K), bf16(r, K)
    xd = g.dev(x).repeat(MOST // PERIOD, 1)
    for act in (MXFP8, T16):
        q, c = bytes_(g, MOST * (32 if act == MXFP8 else 128)), bytes_(g, MOST * 16)
        y = out16(g, MOST, K)
        mx.mx_add_rms_norm(MOST, K, xd, K, None, 0, g.dev(w), 1e-6, act, 0, None, 0, y, K, q, K, c,
                           1)
        torch.cuda.synchronize()
        assert same_as_first(y)
        first = g.host_u16(y[:PERIOD])
        check_norm((None, first, None, None), x, None, w, 1e-6, BF16, 0)
        oq, oc = oracle.quant_act(first, 0)
        if act == MXFP8:
            assert same_as_first(q) and np.array_equal(q[:PERIOD * K].cpu().numpy(), oq.ravel())
            assert same_as_first(c[:MOST])
            assert np.array_equal(c[:PERIOD].cpu().numpy(), oc.ravel())
            assert bool((c[MOST:] == 0xAB).all())
        else:
            last = MOST // 16 - 1                         # the last tile: rows 984 .. 999
            hq, hc = g.t16_unpack(q[last * 2048:].cpu().numpy(), c[last * 256:].cpu().numpy(), 16,
                                  K)
            assert np.array_equal(hq[:, :K], oq[-16:]) and np.array_equal(hc[:, :1], oc[-16:])


@pytest.mark.parametrize("E,topk", [(1024, 8), (3, 1), (1, 1)])
def test_sort_of_the_most_pairs(g, mx, E, topk):
    import torch
    r = rng(111, E)
    ids = r.integers(-1, E + 1, (MOST // topk, topk)).astype(np.int32)
    off = torch.full((E + 1,), -7, dtype=torch.int32, device=g.DEV)
    rows, pos = (torch.full((MOST + 1,), -7, dtype=torch.int32, device=g.DEV) for _ in range(2))
    need = mx.mx_moe_sort_workspace(E, MOST // topk, topk)
    mx.mx_moe_sort(E, MOST // topk, topk, g.dev(ids), off, rows, pos, bytes_(g, need), need)
    torch.cuda.synchronize()
    assert int(rows[-1]) == -7 and int(pos[-1]) == -7
    want = ref.sort(ids, E)
    for got, exact in zip((off, rows[:-1], pos[:-1]), want):
        assert np.array_equal(got.cpu().numpy(), exact.ravel())


@pytest.mark.parametrize("elem", [0, 1])
def test_grouped_of_the_most_rows(g, mx, elem):
    """Rows gathered from one period of source rows, by three experts and behind
    them rows that none takes."""
    import torch
    E, N, K = 3, 48, 160
    r = rng(112, elem)
    w, codes, packed = weight(g, r, elem, 0, E, N, K)
    W = ref.weights(elem, 0, E, N, K, w, codes)
    x = wl.activations(r, (PERIOD, K), 0.01)
    a = ref.activations(*oracle.quant_act(x, 0))
    off = np.array([0, 1300013, 1300014, 3999001], np.int32)
    rows = torch.arange(MOST, dtype=torch.int32, device=g.DEV) % PERIOD
    y = out16(g, MOST, N)
    need = mx.mx_grouped_workspace(elem, 0, E, N, K, MOST, 1, 0)
    mx.mx_grouped_linear(elem, 0, E, N, K, *packed, MOST, g.dev(off), MXFP8, 0, PERIOD, g.dev(x), K,
                         None, 0, None, 0, rows, 0, y, N, bytes_(g, need, fill=0x7F), need)
    torch.cuda.synchronize()
    assert bool((y[int(off[-1]):] == NAN16).all())
    for e in range(E):
        out, tol = ref.grouped(a, W[e:e + 1], [0, PERIOD], 0)
        got = y[int(off[e]):int(off[e + 1])]
        first = int(off[e]) % PERIOD
        pad = torch.zeros(-len(got) % PERIOD, N, dtype=got.dtype, device=got.device)
        full = torch.cat([got, pad]).view(torch.bfloat16).double().view(-1, PERIOD, N)
        dev = lambda v: torch.from_numpy(np.roll(v, -first, 0)).to(g.DEV)  # noqa: E731
        near = (full - dev(out)).abs() <= dev(tol) + 2.0 ** -133
        assert bool(near.view(-1, N)[:len(got)].all()), e


def test_combine_of_the_most_tokens(g, mx):
    import torch
    N, M = 24, 77
    r = rng(113)
    ys = bf16(r, M, N)
    pos = r.integers(-1, M + 1, (PERIOD, 1)).astype(np.int32)
    wts = r.standard_normal((PERIOD, 1)).astype(np.float32)
    y = out16(g, MOST, N)
    mx.mx_moe_combine(MOST, 1, N, M, g.dev(ys), N, g.dev(pos).repeat(MOST // PERIOD, 1),
                      g.dev(wts).repeat(MOST // PERIOD, 1), y, N)
    torch.cuda.synchronize()
    assert same_as_first(y)
    ref.assert_within(g.host_u16(y[:PERIOD]), *ref.combine(ys, pos, wts), "combine")


@pytest.mark.parametrize("invariant", [False, True])
def test_adapters_of_the_most_rows(g, mx, invariant):
    import torch
    L, R, N, K = 4, 8, 32, 64
    a, b, s, x, ids, base = lora_inputs(rng(114), L, R, N, K, PERIOD, "mixed")
    rep = lambda v: g.dev(v).repeat(*([MOST // PERIOD] + [1] * (v.ndim - 1)))  # noqa: E731
    y = out16(g, MOST, N)
    before = mx.mx_set_batch_invariant(invariant)
    try:
        need = mx.mx_lora_workspace(L, R, N, K, MOST)
        mx.mx_lora_add(L, R, N, K, g.dev(a), g.dev(b), g.dev(s), MOST, rep(x), K, rep(ids),
                       rep(base), N, y, N, bytes_(g, need, fill=0xFF), need)
        torch.cuda.synchronize()
    finally:
        mx.mx_set_batch_invariant(before)
    assert same_as_first(y)
    ref.assert_within(g.host_u16(y[:PERIOD]), *ref.lora(x, a, b, s, ids, base), "lora")


@pytest.mark.parametrize("M", [300, 7200])
@pytest.mark.parametrize("epi", [0, 1])
def test_grouped_far_experts(g, mx, M, epi):
    """More than 2^32 bytes of weights, rows on the last two experts only: the
    streaming form (300 rows of y) and the tiled one (7200)."""
    import torch
    E, N, K = 1024, 1056, 4096
    r = rng(115, M)
    w, codes, packed = weight(g, r, 0, 0, 2, N, K)
    W = ref.weights(0, 0, 2, N, K, w, codes)
    wb, cb = mx.mx_packed_sizes(0, 0, E, N, K)
    assert wb > 2 ** 32
    wp, cp = bytes_(g, wb, fill=0x7F), bytes_(g, cb, fill=0x80)
    wp[-packed[0].numel():] = packed[0]
    cp[-packed[1].numel():] = packed[1]
    x = wl.activations(r, (300, K), 0.01)
    off = np.zeros(E + 1, np.int32)
    off[-2:] = 41, 300
    width = N // 2 if epi else N
    y = out16(g, M, width)
    qb, cbx = mx.mx_act_t16_sizes(M, K)
    q, c = bytes_(g, qb, fill=0x7F), bytes_(g, cbx, fill=127)
    q1, c1 = g.quant_t16(x, 0)
    q[:q1.numel()], c[:c1.numel()] = q1, c1
    mx.mx_grouped_linear(0, 0, E, N, K, wp, cp, M, g.dev(off), T16, 0, 0, None, 0, q, 0, c, 0, None,
                         epi, y, width, None, 0)
    torch.cuda.synchronize()
    assert bool((y[300:] == NAN16).all())
    a = ref.activations(*oracle.quant_act(x, 0))
    check_grouped(g.host_u16(y[:300]), a, W, [0, 41, 300], epi)


def test_grouped_far_output_rows(g, mx):
    """Rows of y and of the staged activation beyond 2^32 bytes."""
    import torch
    E, N, K, ldy, M = 2, 32, 2048, 8192, 2200000           # 36 GB of y, 4.5 GB staged
    r = rng(116)
    w, codes, packed = weight(g, r, 0, 1, E, N, K)
    W = ref.weights(0, 1, E, N, K, w, codes)
    x = wl.activations(r, (7, K), 0.01)
    a = ref.activations(*oracle.quant_act(x, 0))
    rows = torch.full((M,), -1, dtype=torch.int32, device=g.DEV)
    last = torch.tensor([0, 1, 1100000, 1100001, M - 17, M - 2, M - 1], device=g.DEV)
    rows[last] = torch.arange(7, dtype=torch.int32, device=g.DEV)
    off = np.array([0, 1100001, M], np.int32)
    y = torch.full((M, ldy), NAN16, dtype=torch.int16, device=g.DEV)
    need = mx.mx_grouped_workspace(0, 1, E, N, K, M, 1, 0)
    assert need > 2 ** 32
    ws = bytes_(g, need)
    mx.mx_grouped_linear(0, 1, E, N, K, *packed, M, g.dev(off), MXFP8, 0, 7, g.dev(x), K, None, 0,
                         None, 0, rows, 0, y, ldy, ws, need)
    torch.cuda.synchronize()
    got = g.host_u16(y[last, :N])
    out0, tol0 = ref.grouped(a, W[:1], [0, 7], 0)
    out1, tol1 = ref.grouped(a, W[1:], [0, 7], 0)
    first = np.arange(7)[:, None] < 3
    ref.assert_within(got, np.where(first, out0, out1), np.where(first, tol0, tol1), "far rows")
    rest = torch.ones(M, dtype=torch.bool, device=g.DEV)
    rest[last] = False
    assert bool(((y[:, :N][rest] & 0x7FFF) == 0).all())     # no source row: zeros
    assert bool((y[:, N:N + 8] == NAN16).all())


# ---- the longest rows ---------------------------------------------------------------
# Few values are not zero and every result is one product or a short sum, so the
# definitions need no long sums: the cases test where things are read and written.


def sparse16(g, rows, cols, at, values):
    """A device bf16 buffer of zeros with values[m][i] in column at[i] of row m."""
    import torch
    t = torch.zeros(rows, cols, dtype=torch.int16, device=g.DEV)
    t[:, torch.from_numpy(np.asarray(at)).to(g.DEV)] = g.dev(values)
    return t


@pytest.mark.parametrize("M", [2, 513])
def test_adapters_of_the_longest_rows(g, mx, M):
    import torch
    L, R, N, K = 2, 8, 16, 16777184 if M == 2 else 1048608
    r = rng(120, M)
    at = np.array([0, 1, K // 2, K - 33, K - 1])
    av, xv, b = bf16(r, L * R, 5), bf16(r, M, 5), bf16(r, L, N, R)
    a, x = sparse16(g, L * R, K, at, av), sparse16(g, M, K, at, xv)
    ids, base = np.arange(M, dtype=np.int32) % 3, bf16(r, M, N)
    y = out16(g, M + 1, N)
    need = mx.mx_lora_workspace(L, R, N, K, M)
    mx.mx_lora_add(L, R, N, K, a, g.dev(b), None, M, x, K, g.dev(ids), g.dev(base), N, y, N,
                   bytes_(g, need, fill=0xFF), need)
    torch.cuda.synchronize()
    out, tol = ref.lora(xv, av.reshape(L, R, 5), b, None, ids, base)
    ref.assert_within(g.host_u16(y[:M]), out, tol, "long adapters")
    assert bool((y[M:] == NAN16).all())


@pytest.mark.parametrize("M", [3, 512])
def test_adapters_of_the_widest_output(g, mx, M):
    """As many columns as a call takes; at 512 rows as many as keep the buffers
    in some gigabytes."""
    import torch
    L, R, N, K = 2, 8, 16776960 if M == 3 else 1048592, 32
    r = rng(121, M)
    at = np.array([0, 255, 256, N // 2, N - 257, N - 1])
    a, bv, x = bf16(r, L, R, K), bf16(r, L, 6, R), bf16(r, M, K)
    b = torch.zeros(L, N, R, dtype=torch.int16, device=g.DEV)
    b[:, torch.from_numpy(at).to(g.DEV)] = g.dev(bv)
    ids = np.arange(M, dtype=np.int32) % 3 - 1
    base = torch.full((M, N), 0x3F80, dtype=torch.int16, device=g.DEV)
    y = out16(g, M + 1, N)
    need = mx.mx_lora_workspace(L, R, N, K, M)
    mx.mx_lora_add(L, R, N, K, g.dev(a), b, None, M, g.dev(x), K, g.dev(ids), base, N, y, N,
                   bytes_(g, need, fill=0xFF), need)
    torch.cuda.synchronize()
    out, tol = ref.lora(x, a, bv, None, ids, np.full((M, 6), 0x3F80, np.uint16))
    ref.assert_within(g.host_u16(y[:M, torch.from_numpy(at).to(g.DEV)]), out, tol, "wide adapters")
    y[:M, torch.from_numpy(at).to(g.DEV)] = 0x3F80
    assert bool((y[:M] == 0x3F80).all()) and bool((y[M:] == NAN16).all())


def test_combine_of_the_widest_rows(g, mx):
    import torch
    N, M, T = 134215680, 3, 2
    r = rng(122)
    at = np.array([0, 2047, 2048, N // 2, N - 2049, N - 1])
    yv = bf16(r, M, 6)
    ys = sparse16(g, M, N, at, yv)
    pos, wts = np.array([[2, 0], [1, 3]], np.int32), r.standard_normal((T, 2)).astype(np.float32)
    y = out16(g, T + 1, N)
    mx.mx_moe_combine(T, 2, N, M, ys, N, g.dev(pos), g.dev(wts), y, N)
    torch.cuda.synchronize()
    cols = torch.from_numpy(at).to(g.DEV)
    ref.assert_within(g.host_u16(y[:T, cols]), *ref.combine(yv, pos, wts), "wide combine")
    y[:T, cols] = 0
    assert bool((y[:T] & 0x7FFF == 0).all()) and bool((y[T:] == NAN16).all())


@pytest.mark.parametrize("elem", [0, 1])
@pytest.mark.parametrize("M", [3, 520])
def test_grouped_of_the_longest_rows(g, mx, M, elem):
    """One expert, K as long as 272 token rows allow in 32-bit offsets (with 520
    rows a shorter one, for the tiled form)."""
    import torch
    N, K = 16, 7895040 if M == 3 else 1048608
    r = rng(123, M, elem)
    at = np.array([0, 1, K // 2, K - 33, K - 1])          # columns of K that hold values
    # e4m3 1.0 = 0x38; e2m1 1.0 = 2 in either nibble; codes 127: a product is one value
    w = torch.zeros(N, K if elem == 0 else K // 2, dtype=torch.uint8, device=g.DEV)
    hot = np.arange(N) % 5
    for n in range(N):
        k = int(at[hot[n]])
        if elem == 0:
            w[n, k] = 0x38
        else:
            w[n, k // 2] = 0x20 if k % 2 else 0x02
    codes = torch.full((N, K // 32), 127, dtype=torch.uint8, device=g.DEV)
    wb, cb = mx.mx_packed_sizes(elem, 0, 1, N, K)
    wp, cp, ws = bytes_(g, wb), bytes_(g, cb), bytes_(g, 256)
    mx.mx_pack_weights(elem, 0, 1, N, K, w, codes, wp, cp, ws, 256)
    xv = np.full((M, 5), 0x3F80, np.uint16)               # 1.0, and a row's own sign pattern
    xv[r.random((M, 5)) < 0.5] = 0xBF80
    x = sparse16(g, M, K, at, xv)
    y = out16(g, M + 1, N)
    need = mx.mx_grouped_workspace(elem, 0, 1, N, K, M, 1, 0)
    ws = bytes_(g, need, fill=0x7F)
    mx.mx_grouped_linear(elem, 0, 1, N, K, wp, cp, M, g.dev(np.array([0, M], np.int32)), MXFP8, 0,
                         M, x, K, None, 0, None, 0, None, 0, y, N, ws, need)
    torch.cuda.synchronize()
    # (columns 0 and 1 share a block, as do the last two of five: all are +-1 there,
    # which the block's scale holds exactly)
    assert np.array_equal(g.host_u16(y[:M]), xv[:, hot])
    assert bool((y[M:] == NAN16).all())


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("epi", [0, 1])
def test_grouped_of_the_widest_output(g, mx, M, epi):
    import torch
    E, N, K = 1, 4194288, 32
    r = rng(124, M)
    w, codes, _ = weight(g, r, 0, 0, E, 64, K)
    W = ref.weights(0, 0, E, 64, K, w, codes)
    # the 64 weight rows over and over: 65535.75 times
    reps = -(-N // 64)
    wd = g.dev(w.reshape(64, K)).repeat(reps, 1)[:N].contiguous()
    cd = g.dev(codes.reshape(64, 1)).repeat(reps, 1)[:N].contiguous()
    wb, cb = mx.mx_packed_sizes(0, 0, E, N, K)
    wp, cp, ws = bytes_(g, wb), bytes_(g, cb), bytes_(g, 256)
    mx.mx_pack_weights(0, 0, E, N, K, wd, cd, wp, cp, ws, 256)
    x = wl.activations(r, (M, K), 0.01)
    width, period = (N // 2, 32) if epi else (N, 64)
    y = out16(g, M + 1, width)
    need = mx.mx_grouped_workspace(0, 0, E, N, K, M, 1, 0)
    mx.mx_grouped_linear(0, 0, E, N, K, wp, cp, M, g.dev(np.array([0, M], np.int32)), MXFP8, 0, M,
                         g.dev(x), K, None, 0, None, 0, None, epi, y, width, bytes_(g, need), need)
    torch.cuda.synchronize()
    whole = width // period * period
    v = y[:M, :whole].view(M, -1, period)
    assert torch.equal(v, v[:, :1].expand_as(v))
    assert torch.equal(y[:M, whole:], y[:M, :width - whole]) and bool((y[M:] == NAN16).all())
    a = ref.activations(*oracle.quant_act(x, 0))
    out, tol = ref.grouped(a, W, [0, M], epi)
    ref.assert_within(g.host_u16(y[:M, :period]), out, tol, "wide grouped")
