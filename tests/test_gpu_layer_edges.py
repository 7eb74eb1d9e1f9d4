"""Edges of the operators between a layer's products that need cases of their own:
gates and weights that are not finite."""
import numpy as np
import pytest

from test_gpu_layer import (MXFP8, NAN16, block_inputs, check_block, g, mx, rng,  # noqa: F401
                            run_block)

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
