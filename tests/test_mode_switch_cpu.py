"""A call reads the batch-invariant mode once: another thread that changes the
mode between the check of the workspace and the launch (played by stand-ins
that change it at exactly that point) cannot make the launch write more than
the checked size.  On a host-only build of the library's host code."""
import ctypes as C
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import microscaling_quantized_linear_amd as mx  # noqa: E402


def A(i):
    """Fake, distinct, 256-byte aligned device addresses: never dereferenced."""
    return (i + 1) << 40


@pytest.fixture(scope="module")
def host_lib(tmp_path_factory):
    csrc = os.path.join(ROOT, "microscaling_quantized_linear_amd", "csrc")
    lib = str(tmp_path_factory.mktemp("mode") / "libmx_mode.so")
    src = [os.path.join(csrc, f) for f in ("mx_api.cpp", "mx_ops_api.cpp")]
    src += [os.path.join(ROOT, "tests", "sanitize", f)
            for f in ("host_stubs.cpp", "mode_stubs.cpp")]
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include", *src, "-o", lib], capture_output=True, text=True)
    if r.returncode != 0 and "hip_runtime.h" in r.stderr:
        pytest.skip("HIP headers not found")
    assert r.returncode == 0, r.stderr[-3000:]
    return lib


def child(lib, what):
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib, what], capture_output=True,
                       text=True, env=dict(os.environ, MX_LOG="1"), timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert f"{what} ok" in r.stdout
    return r.stderr


def test_adapters(host_lib):
    child(host_lib, "adapters")


def _adapters(L):
    switch, written = C.c_int.in_dll(L, "mx_switch_to"), C.c_long.in_dll(L, "mx_lora_written")
    need, M = C.c_size_t(), 4096
    for before, after in ((1, 0), (0, 1)):
        switch.value = -1
        L.mx_set_batch_invariant(before)
        assert L.mx_lora_workspace(8, 64, 4096, 7168, M, C.byref(need)) == 0
        switch.value = after
        status = L.mx_lora_add(8, 64, 4096, 7168, A(0), A(1), None, M, A(2), 7168, A(3), A(4),
                               4096, A(5), 4096, A(6), need.value, None)
        assert status == 0 and written.value == need.value, (before, status, written.value)


def test_linear(host_lib):
    """The workspace of a pre-quantized prompt is 0 with the mode on, where the
    GEMV reads the rows as they are, and a restaged copy with it off."""
    lines = [ln for ln in child(host_lib, "linear").splitlines() if ln.startswith("mx: linear")]
    assert len(lines) == 2 and "gemv" in lines[0] and "gemm_w8a8_kernel" in lines[1], lines


def _linear(L):
    switch, need, M = C.c_int.in_dll(L, "mx_switch_to"), C.c_size_t(), 100
    for before in (1, 0):
        switch.value = -1
        L.mx_set_batch_invariant(before)
        assert L.mx_linear_workspace(0, 0, 512, 1024, M, 1, 1, C.byref(need)) == 0
        assert (need.value == 0) == (before == 1)
        switch.value = 1 - before
        status = L.mx_linear(0, 0, 512, 1024, A(0), A(1), M, 1, 0, None, 0, A(2), 1024, A(3), 32,
                             None, A(4), 512, A(5) if need.value else None, need.value, None)
        assert status == 0


if __name__ == "__main__":
    mx.LIB_PATH = sys.argv[1]
    {"adapters": _adapters, "linear": _linear}[sys.argv[2]](mx.lib())
    print(sys.argv[2], "ok")
