"""The dispatch trace of mx_linear_epilogue names the launch that runs: waves, steps
and tiles, on a host-only build of the library's host code whose launchers count.
The tuning overrides of mx_linear's launch shapes do not change it."""
import ast
import ctypes as C
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import microscaling_quantized_linear_amd as mx  # noqa: E402

BF16, MXFP8, T16 = 0, 1, 2


def A(i):
    """Fake, distinct, 256-byte aligned device addresses: never dereferenced."""
    return (i + 1) << 40


SHAPES = [  # elem, M, N, K, waves, steps, tiles of the bf16 GEMV with an epilogue
    (1, 4, 4096, 4096, 8, 4, 1), (0, 16, 4096, 7168, 8, 4, 1), (1, 4, 4112, 4096, 8, 4, 2),
    (0, 17, 4096, 4096, 8, 4, 2), (0, 17, 2048, 4096, 8, 4, 1),
    (0, 4, 8192, 2048, 4, 4, 1), (1, 8, 4096, 1568, 2, 8, 1), (0, 8, 4096, 512, 2, 2, 1),
    (0, 1, 64, 96, 1, 2, 1)]


@pytest.fixture(scope="module")
def host_lib(tmp_path_factory):
    csrc = os.path.join(ROOT, "microscaling_quantized_linear_amd", "csrc")
    lib = str(tmp_path_factory.mktemp("trace") / "libmx_trace.so")
    src = [os.path.join(csrc, f) for f in ("mx_api.cpp", "mx_plan.cpp")]
    src.append(os.path.join(ROOT, "tests", "sanitize", "host_stubs.cpp"))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include", *src, "-o", lib], capture_output=True, text=True)
    if r.returncode != 0 and "hip_runtime.h" in r.stderr:
        pytest.skip("HIP headers not found")
    assert r.returncode == 0, r.stderr[-3000:]
    return lib


def trace(lib, calls, **env):
    """The trace's lines of the calls (elem, layout, M, N, K, act, form), in a process of
    its own: the environment is read once."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib, repr(calls)],
                       capture_output=True, text=True, env=dict(os.environ, MX_LOG="1", **env),
                       timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("mx: linear: ") and "gem" in ln]
    assert len(lines) == len(calls)
    return lines


@pytest.mark.parametrize("env", [{}, dict(MX_GEMV_WAVES="1", MX_GEMV_CHUNK="8", MX_GEMV_TILES="4")],
                         ids=["plain", "overridden"])
def test_gemv_shapes(host_lib, env):
    lines = trace(host_lib, [(e, 0, M, N, K, BF16, "x") for e, M, N, K, *_ in SHAPES], **env)
    for line, (_, M, N, K, nw, steps, tiles) in zip(lines, SHAPES):
        assert "gemv_kernel" in line and "with epilogue" in line
        assert f"{nw} waves x {steps}-step chunks x {tiles} tiles; M={M} N={N} K={K}" in line, line


def test_larger_forms(host_lib):
    """The sizes that test the products' larger forms on the GPU reach them."""
    from test_gpu_layer_edges import LARGER
    lines = trace(host_lib, [(0, layout, M, N, K, act, form) for layout, M, N, K, act, form, *_ in LARGER])
    for line, (*_, kernel, plan) in zip(lines, LARGER):
        assert f"{kernel} " in line and f"{plan}; " in line, line


def _calls(path, calls):
    """In the child process: each call, fn SiLU, no residual."""
    mx.LIB_PATH = path
    L = mx.lib()
    for elem, layout, M, N, K, act, form in calls:
        given = form != "x"
        need = C.c_size_t()
        assert L.mx_linear_workspace(elem, layout, N, K, M, act, int(given), C.byref(need)) == 0
        st = L.mx_linear_epilogue(elem, layout, N, K, A(0), A(1), M, act, 0,
                                  None if given else A(2), K, A(3) if given else None, K,
                                  A(4) if given else None, K // 32, None, 3, 0, None, 0, A(5), N,
                                  A(6), need.value, None)
        assert st == 0, (st, M, N, K)


if __name__ == "__main__":
    _calls(sys.argv[1], ast.literal_eval(sys.argv[2]))
