"""The tiled form of the grouped product at every kind of tile: 256- and 128-row
tiles side by side, remainders on both sides of every border, K with and without
a cut last step and a remainder of steps, each weight form, with and without
SiLU.  Which form serves a shape is read from the dispatch trace, so a change of
the rule cannot leave these cases to another kernel unnoticed."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "tests")):
    if path not in sys.path:
        sys.path.insert(0, path)
import ops_ref as ref  # noqa: E402
import oracle  # noqa: E402
from microscaling_quantized_linear_amd import workloads as wl  # noqa: E402
from test_gpu_ops import FORMS, check_grouped, g, mx, rng, run_grouped, weight  # noqa: E402,F401
from test_gpu_ops import SHAPES as OPS_SHAPES  # noqa: E402

pytestmark = pytest.mark.gpu

LONG = [0, 1, 127, 128, 129, 255, 256, 257, 383, 384, 385, 20, 64, 65, 130, 140]
SHORT = [0, 1, 63, 64, 65, 127, 128, 129, 15, 16, 17, 48, 200, 257, 33, 90]
# (E, N, K, rows an expert in turn, tile form)
SHAPES = [
    (64, 1056, 544, LONG, 256),      # a cut last step, five steps
    (130, 288, 1024, LONG, 256),     # eight steps
    (86, 544, 2048, LONG, 256),      # sixteen steps
    (130, 288, 1056, LONG, 256),     # nine steps, the last cut
    (130, 288, 1408, LONG, 256),     # eleven steps
    (130, 288, 1024, SHORT, 128),
    (70, 544, 2048, SHORT, 128),
    (130, 288, 1408, SHORT, 128),
]


def offsets_of(E, counts, key):
    n = [counts[i % len(counts)] for i in range(E)]
    return np.concatenate([[0], np.cumsum(rng(90, key).permutation(n))]).astype(np.int32)


def rows_of(E, counts):
    """Rows of y: seven behind the last expert's."""
    return int(offsets_of(E, counts, 0)[-1]) + 7


@pytest.mark.parametrize("elem,layout", FORMS)
@pytest.mark.parametrize("E,N,K,counts,tile", SHAPES,
                         ids=[f"{E}x{N}x{K}-{tile}" for E, N, K, _, tile in SHAPES])
def test_tiles(g, mx, E, N, K, counts, tile, elem, layout):
    r = rng(91, E, N, K, elem, layout)
    w, codes, packed = weight(g, r, elem, layout, E, N, K)
    W = ref.weights(elem, layout, E, N, K, w, codes)
    offsets, M = offsets_of(E, counts, K), rows_of(E, counts)
    x = wl.activations(r, (M, K), 0.01)
    a = ref.activations(*oracle.quant_act(x, 0))
    for epi in (0, 1):
        y = run_grouped(g, mx, elem, layout, E, N, K, packed, offsets, M, x=x, epi=epi, pad=8)
        check_grouped(y, a, W, offsets, epi, f"epi {epi}")


def forms_of(calls):
    """The kernel that the dispatch trace names for each (elem, layout, E, N, K, M)."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), repr(calls)],
                       capture_output=True, text=True, env=dict(os.environ, MX_LOG="1"),
                       timeout=110)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    names = re.findall(r"mx: grouped: (grouped_\w+(?: \d+-row tiles)?) ", r.stderr)
    assert len(names) == len(calls), r.stderr[-3000:]
    return names


def test_forms(g):
    calls = [(elem, layout, E, N, K, rows_of(E, counts))
             for E, N, K, counts, _ in SHAPES for elem, layout in FORMS]
    want = [f"grouped_gemm_kernel {tile}-row tiles" for *_, tile in SHAPES for _ in FORMS]
    # test_gpu_ops.py's shape for the 256-row tiles
    calls.append((0, 0, *OPS_SHAPES[-1][:4]))
    want.append("grouped_gemm_kernel 256-row tiles")
    assert forms_of(calls) == want


def test_form_of_few_weight_panels(g):
    """Fewer weight panels than half the compute units: streamed while that takes
    less than one tile does, up to about 90 panel batches of 64 rows; 16 rows an
    expert always."""
    stream, tiled = "grouped_stream_kernel", "grouped_gemm_kernel 128-row tiles"
    cases = [  # E, N, rows an expert, form
        (8, 3840, 8, stream), (8, 3840, 16, stream), (8, 3840, 64, tiled), (8, 3840, 128, tiled),
        (8, 3840, 190, tiled), (12, 2048, 16, stream), (12, 2048, 64, tiled),
        (8, 2048, 64, stream), (8, 2048, 128, tiled), (6, 2048, 64, stream), (6, 2048, 96, tiled),
        (8, 1024, 128, stream), (8, 1024, 192, tiled), (1, 4096, 192, stream),
        (1, 4096, 256, tiled), (1, 256, 150, stream), (1, 256, 300, tiled)]
    calls = [(elem, layout, E, N, 512, E * rows) for E, N, rows, _ in cases
             for elem, layout in FORMS]
    assert forms_of(calls) == [form for *_, form in cases for _ in FORMS]


def _trace(calls):
    """In a child process with the trace on: each call, without a row to compute."""
    import torch

    import microscaling_quantized_linear_amd as mx
    for elem, layout, E, N, K, M in calls:
        zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        w, c = map(zeros, mx.mx_packed_sizes(elem, layout, E, N, K))
        q, qc = map(zeros, mx.mx_act_t16_sizes(M, K))
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        mx.mx_grouped_linear(elem, layout, E, N, K, w, c, M, off, 2, 0, 0, None, 0, q, 0, qc, 0,
                             None, 0, y, N, None, 0)
        torch.cuda.synchronize()


if __name__ == "__main__":
    import ast
    _trace(ast.literal_eval(sys.argv[1]))
