"""Edges of the operators around the linear that need cases of their own:
rows that are not finite, tile forms and remainders, buffers that share a row."""
import numpy as np
import pytest

import oracle
from test_gpu_ops import BF16, MXFP8, T16, bf16, check_norm, g, mx, rng, run_norm  # noqa: F401

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
