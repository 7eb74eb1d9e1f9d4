"""Edges of the operators around the linear that need cases of their own:
rows that are not finite, tile forms and remainders, buffers that share a row."""
import numpy as np
import pytest

import ops_ref as ref
from microscaling_quantized_linear_amd import workloads as wl
from test_gpu_ops import (BF16, MXFP8, NAN16, T16, Layer, bf16, bytes_, check_norm,  # noqa: F401
                          g, lora_inputs, mx, rng, run_grouped, run_lora, run_norm, split, weight)

pytestmark = pytest.mark.gpu


def odd_rows(K):
    """x [5, K] for a norm with eps 0: a zero row (its y is NaN), a row with a
    NaN, one with both infinities, and two ordinary rows."""
    x = bf16(rng(70, K), 5, K)
    x[0] = 0
    x[1, K // 2] = 0x7FC0
    x[3, 1], x[3, K - 1] = 0x7F80, 0xFF80
    return x, bf16(rng(71, K), K)


# ---- residual norm ----------------------------------------------------------------


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("K", [96, 544, 1056])
def test_norm_padding_of_rows_that_are_not_finite(g, mx, K, rule):
    """T16: zeros with code 127 past K (run_norm checks every byte of it), the
    ordinary rows as ever, the codes those of a stored y."""
    x, w = odd_rows(K)
    s, y, q, c = run_norm(g, mx, x, None, w, 0.0, T16, rule)
    assert ((y[:2] & 0x7FFF) > 0x7F80).all()
    for m in (2, 4):
        row = slice(m, m + 1)
        check_norm((s[row], y[row], q[row], c[row]), x[row], None, w, 0.0, T16, rule)
    xq, xc = g.quant_t16(y, rule)
    _, want = g.t16_unpack(xq.cpu().numpy(), xc.cpu().numpy(), 5, K)
    assert np.array_equal(c, want[:5, :K // 32])


@pytest.mark.parametrize("act", [MXFP8, T16])
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("K", [96, 544, 4128, 7168])
def test_norm_bytes_of_rows_that_are_not_finite(g, mx, K, rule, act):
    """The bytes and codes are the quantization call's of the stored y, also for
    rows of NaN and rows whose infinite y comes from a large weight."""
    x, w = odd_rows(K)
    w[3], w[K - 2] = 0x7F00, 0xFF00                       # +-2^127: y of 2 and more is infinite
    x[4, 3], x[4, K - 2] = 0x4040, 0xC040
    s, y, q, c = run_norm(g, mx, x, None, w, 0.0, act, rule)
    assert ((y[:2] & 0x7FFF) > 0x7F80).all() and (y[4, [3, K - 2]] == 0x7F80).all()
    if act == T16:
        xq, xc = g.quant_t16(y, rule)
        wq, wc = g.t16_unpack(xq.cpu().numpy(), xc.cpu().numpy(), 5, K)
        wq, wc = wq[:5, :K], wc[:5, :K // 32]
    else:
        wq, wc = g.quant(y, rule)
    assert np.array_equal(c, wc) and np.array_equal(q, wq)


# ---- adapters -----------------------------------------------------------------------


@pytest.mark.parametrize("R", [8, 24, 64, 72])
@pytest.mark.parametrize("M", [20, 600])
def test_adapters_beyond_the_range(g, mx, M, R):
    """Finite inputs whose products leave fp32's range: infinities of the result's
    sign (no sum here holds both signs), not NaN; the columns beside them are as
    ever."""
    L, N, K = 5, 64, 96
    a, b, s, x, ids, base = lora_inputs(rng(72, M, R), L, R, N, K, M, "each")
    # A in [1, 2), x in [2^8, 2^9): v beyond 2^13, its remainder's products overflow too
    a, x = a & 0x007F | 0x3F80, x & 0x007F | 0x4380
    b = b & 0x7FFF | 0x0080
    up, down = np.arange(1, N, 7), np.arange(3, N, 7)
    out, tol = ref.lora(x, a, b, s, ids, base)
    b[:, up], b[:, down] = 0x7F00, 0xFF00                 # +-2^127
    y = run_lora(g, mx, a, b, s, x, ids, base)
    assert (y[:, up] == 0x7F80).all() and (y[:, down] == 0xFF80).all()
    rest = np.setdiff1d(np.arange(N), np.concatenate([up, down]))
    ref.assert_within(y[:, rest], out[:, rest], tol[:, rest], "lora")


# ---- column ranges of one wide buffer -----------------------------------------------


def wide(g, rows, cols, **parts):
    """A device buffer [rows, cols] of NaN with arrays in its columns, by their
    first column; returns the buffer and column views (tensors)."""
    buf = np.full((rows, cols), NAN16, np.uint16)
    for name, (at, a) in parts.items():
        if a is not None:
            buf[:a.shape[0], at:at + a.shape[1]] = a
    buf = g.dev(buf)
    return buf, {name: buf[:, at:] for name, (at, _) in parts.items()}


@pytest.mark.parametrize("M", [3, 700])
def test_norm_in_columns_of_one_buffer(g, mx, M):
    """x, the residual, the sum and y side by side: the separate buffers' values,
    and nothing between them written."""
    import torch
    K = 96
    r = rng(80, M)
    x, res, w = bf16(r, M, K), bf16(r, M, K), bf16(r, K)
    want = run_norm(g, mx, x, res, w, 1e-6, BF16, 0)
    buf, v = wide(g, M, 424, x=(0, x), s=(96, None), res=(192, res), y=(320, None))
    mx.mx_add_rms_norm(M, K, v["x"], 424, v["res"], 424, g.dev(w), 1e-6, BF16, 0, v["s"], 424,
                       v["y"], 424, None, 0, None, 0)
    torch.cuda.synchronize()
    h = g.host_u16(buf)
    assert np.array_equal(h[:, :96], x) and np.array_equal(h[:, 192:288], res)
    assert np.array_equal(h[:, 96:192], want[0]) and np.array_equal(h[:, 320:416], want[1])
    assert (h[:, 288:320] == NAN16).all() and (h[:, 416:] == NAN16).all()


@pytest.mark.parametrize("M", [20, 600])
def test_adapters_in_columns_of_one_buffer(g, mx, M):
    """x, base and y side by side."""
    import torch
    L, R, N, K = 5, 24, 80, 96
    a, b, s, x, ids, base = lora_inputs(rng(81, M), L, R, N, K, M, "mixed")
    want = run_lora(g, mx, a, b, s, x, ids, base)
    buf, v = wide(g, M, 264, x=(0, x), y=(96, None), base=(184, base))
    need = mx.mx_lora_workspace(L, R, N, K, M)
    mx.mx_lora_add(L, R, N, K, g.dev(a), g.dev(b), g.dev(s), M, v["x"], 264, g.dev(ids), v["base"],
                   264, v["y"], 264, bytes_(g, need, fill=0xFF), need)
    torch.cuda.synchronize()
    h = g.host_u16(buf)
    assert np.array_equal(h[:, 96:176], want) and np.array_equal(h[:, :96], x)
    assert np.array_equal(h[:, 184:], base) and (h[:, 176:184] == NAN16).all()


@pytest.mark.parametrize("M", [20, 900])
@pytest.mark.parametrize("epi", [0, 1])
def test_grouped_and_combine_in_columns_of_one_buffer(g, mx, M, epi):
    """The grouped product's x and y side by side, then the combine's ys and y."""
    import torch
    E, N, K = 3, 128, 160
    width = N // 2 if epi else N
    r = rng(82, M)
    w, codes, packed = weight(g, r, 0, 0, E, N, K)
    x, offsets = wl.activations(r, (M, K), 0.01), split(r, M, E, "skew")
    want = run_grouped(g, mx, 0, 0, E, N, K, packed, offsets, M, x=x, epi=epi)
    ld = K + width + width + 24
    buf, v = wide(g, M, ld, x=(0, x), y=(K, None), out=(K + width, None))
    need = mx.mx_grouped_workspace(0, 0, E, N, K, M, MXFP8, 0)
    mx.mx_grouped_linear(0, 0, E, N, K, *packed, M, g.dev(offsets), MXFP8, 0, M, v["x"], ld, None,
                         0, None, 0, None, epi, v["y"], ld, bytes_(g, need), need)
    T, topk = M // 4, 3
    pos = r.integers(-1, M, (T, topk)).astype(np.int32)
    wts = r.random((T, topk)).astype(np.float32)
    mx.mx_moe_combine(T, topk, width, M, v["y"], ld, g.dev(pos), g.dev(wts), v["out"], ld)
    torch.cuda.synchronize()
    h = g.host_u16(buf)
    assert np.array_equal(h[:, K:K + width], want) and np.array_equal(h[:, :K], x)
    out, tol = ref.combine(want, pos, wts)
    ref.assert_within(h[:T, K + width:K + 2 * width], out, tol, "combine")
    assert (h[T:, K + width:] == NAN16).all() and (h[:, K + 2 * width:] == NAN16).all()


# ---- together ---------------------------------------------------------------------


def test_two_streams_at_once(g, mx):
    """Two layers with workspaces of their own, on two streams at the same time."""
    import torch
    layers = [Layer(g, mx, T, key=k) for k, T in enumerate((700, 40))]
    want = []
    for layer in layers:
        layer.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in layer.outputs()])
        for t in layer.outputs():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                layer.run()
    torch.cuda.synchronize()
    for layer, outputs in zip(layers, want):
        layer.check()
        for x, y in zip(layer.outputs(), outputs):
            assert torch.equal(x, y)


def test_captured_prompt(g, mx):
    """Prompt sizes captured: the tiled forms, the sort's two launches and the
    64-row adapters, replayed with other inputs in the same buffers."""
    import torch
    a, b = Layer(g, mx, 1100, key=4), Layer(g, mx, 1100, key=5)
    a.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        a.run()
    first = {k: a.d[k].clone() for k in ("x", "ids", "aid")}
    want = []
    for k in range(2):                                    # eager, with a's and b's inputs
        if k:
            for name in first:
                a.d[name].copy_(b.d[name])
        a.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in a.outputs()])
    for turn in range(4):
        for name in first:
            a.d[name].copy_(b.d[name] if turn % 2 else first[name])
        for t in a.outputs():
            t.zero_()
        b.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.outputs(), want[turn % 2]):
            assert torch.equal(x, y)
    a.x, a.ids, a.aid = b.x, b.ids, b.aid
    a.check()
