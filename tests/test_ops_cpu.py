"""CPU-side tests of the operators around the linear: every refusal that the
header names comes before any device work, with the documented status; the
binding refuses tensors that are not on the current GPU; the same calls run
under AddressSanitizer and UndefinedBehaviorSanitizer on a host-only build."""
import ctypes as C
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import microscaling_quantized_linear_amd as mx  # noqa: E402

OK, NULL, SHAPE, ALIGN, VALUE, UNSUP, DEVICE, WS, LAUNCH = range(9)
BIG = 2 ** 62


def A(i):
    """Fake, distinct, 256-byte aligned device addresses, 1 TiB apart: never dereferenced."""
    return (i + 1) << 40


def norm(**kw):
    a = dict(M=4, K=64, x=A(0), ldx=64, res=A(1), ldr=64, w=A(2), eps=1e-6, act=1, rule=0, sum=A(3),
             lds=64, y=A(4), ldy=64, xq=A(5), ldq=64, xc=A(6), ldc=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_add_rms_norm(*a.values(), None)


def sort(**kw):
    a = dict(E=8, T=4, topk=2, ids=A(0), off=A(1), rows=A(2), pos=A(3), ws=None, wsb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_moe_sort(*a.values(), None)


def grouped(**kw):
    a = dict(elem=0, layout=0, E=4, N=64, K=256, w=A(0), c=A(1), M=20, off=A(2), act=1, rule=0,
             xrows=20, x=A(3), ldx=256, xq=None, ldq=0, xc=None, ldc=0, rows=A(4), epi=0, y=A(5),
             ldy=64, ws=A(6), wsb=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_grouped_linear(*a.values(), None)


def combine(**kw):
    a = dict(T=4, topk=2, N=64, M=8, ys=A(0), ldys=64, pos=A(1), w=A(2), y=A(3), ldy=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_moe_combine(*a.values(), None)


def lora(**kw):
    a = dict(L=3, R=16, N=64, K=96, a=A(0), b=A(1), s=A(2), M=5, x=A(3), ldx=96, ids=A(4),
             base=A(5), ldb=64, y=A(6), ldy=64, ws=A(7), wsb=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_lora_add(*a.values(), None)


REFUSED = [
    # residual norm
    (norm, SHAPE, [dict(M=0), dict(M=4000001), dict(K=48), dict(K=0), dict(K=65568, ldx=65568),
                   dict(ldx=32), dict(ldr=56), dict(lds=32), dict(ldy=32), dict(ldq=48),
                   dict(ldc=1), dict(eps=-1e-6), dict(eps=float("nan")), dict(ldx=BIG),
                   dict(ldq=BIG), dict(M=-1), dict(K=-64)]),
    (norm, NULL, [dict(x=None), dict(w=None), dict(xq=None), dict(xc=None),
                  dict(act=0, y=None), dict(act=2, xc=None)]),
    (norm, ALIGN, [dict(x=A(0) + 8), dict(ldx=68), dict(res=A(1) + 2), dict(ldr=68),
                   dict(w=A(2) + 2), dict(sum=A(3) + 8), dict(lds=66), dict(y=A(4) + 4),
                   dict(ldy=68), dict(xq=A(5) + 8), dict(ldq=72), dict(act=2, xc=A(6) + 4)]),
    (norm, UNSUP, [dict(act=3), dict(rule=2), dict(act=0, rule=5),
                   dict(sum=A(0) + 16), dict(sum=A(0), lds=128),   # on x, displaced
                   dict(sum=A(1) + 128), dict(y=A(3)), dict(sum=A(2)), dict(y=A(2)),
                   dict(xq=A(0)), dict(xq=A(1)), dict(xq=A(3)), dict(xc=A(4)), dict(xc=A(5)),
                   dict(sum=A(0), y=A(0)), dict(act=2, xq=A(2)), dict(act=2, xc=A(5) + 1024)]),
    # sort
    (sort, SHAPE, [dict(E=0), dict(E=1025), dict(T=0), dict(topk=0), dict(topk=9), dict(T=2000001),
                   dict(T=BIG, topk=8), dict(T=-4)]),
    (sort, NULL, [dict(ids=None), dict(off=None), dict(rows=None), dict(pos=None)]),
    (sort, ALIGN, [dict(ids=A(0) + 2), dict(off=A(1) + 1), dict(rows=A(2) + 2),
                   dict(pos=A(3) + 3), dict(T=5000, ws=A(4) + 4, wsb=1 << 20)]),
    (sort, WS, [dict(T=5000), dict(T=5000, ws=A(4), wsb=64)]),
    (sort, UNSUP, [dict(rows=A(0)), dict(pos=A(0) + 16), dict(off=A(2)), dict(pos=A(2)),
                   dict(T=5000, ws=A(0), wsb=1 << 20)]),
    # grouped products
    (grouped, SHAPE, [dict(E=0), dict(E=65536), dict(N=40), dict(N=0), dict(K=100), dict(K=0),
                      dict(M=0), dict(M=4000001), dict(xrows=0), dict(rows=None, xrows=19),
                      dict(ldx=128), dict(ldy=56), dict(epi=1, ldy=24), dict(ldx=BIG),
                      dict(ldy=1 << 24), dict(N=16 * (1 << 40)), dict(K=32 * (1 << 30)),
                      dict(N=1 << 24, K=128, ldx=128, ldy=1 << 24),
                      dict(x=None, xq=A(3), xc=A(7), ldq=240, ldc=8),
                      dict(x=None, xq=A(3), xc=A(7), ldq=256, ldc=7)]),
    (grouped, NULL, [dict(w=None), dict(c=None), dict(off=None), dict(y=None), dict(x=None),
                     dict(x=None, xq=A(3), ldq=256), dict(act=2, rows=None),
                     dict(act=2, rows=None, xq=A(3))]),
    (grouped, ALIGN, [dict(w=A(0) + 8), dict(c=A(1) + 4), dict(off=A(2) + 2), dict(y=A(5) + 8),
                      dict(ldy=68), dict(x=A(3) + 2), dict(ldx=260), dict(rows=A(4) + 1),
                      dict(ws=A(6) + 8), dict(x=None, xq=A(3) + 8, xc=A(7), ldq=256, ldc=8),
                      dict(x=None, xq=A(3), xc=A(7), ldq=264, ldc=8),
                      dict(act=2, rows=None, xq=A(3), xc=A(7) + 4)]),
    (grouped, UNSUP, [dict(elem=2), dict(layout=2), dict(elem=1, layout=1), dict(act=0),
                      dict(act=3), dict(rule=2), dict(epi=2),
                      dict(act=2, xq=A(3), xc=A(7)),          # T16 with an index
                      dict(y=A(3)), dict(y=A(4)), dict(y=A(2)), dict(ws=A(3)), dict(ws=A(4)),
                      dict(ws=A(5)), dict(act=2, rows=None, xq=A(5), xc=A(7))]),
    (grouped, WS, [dict(ws=None), dict(wsb=100)]),
    # combine
    (combine, SHAPE, [dict(T=0), dict(topk=0), dict(N=0), dict(N=60), dict(M=0), dict(ldys=56),
                      dict(ldy=56), dict(T=4000001), dict(T=BIG), dict(ldys=BIG), dict(N=BIG),
                      dict(N=134215688, ldys=134215688, ldy=134215688)]),
    (combine, NULL, [dict(ys=None), dict(pos=None), dict(w=None), dict(y=None)]),
    (combine, ALIGN, [dict(ys=A(0) + 8), dict(ldys=68), dict(pos=A(1) + 2), dict(w=A(2) + 1),
                      dict(y=A(3) + 8), dict(ldy=68)]),
    (combine, UNSUP, [dict(y=A(0)), dict(y=A(1)), dict(y=A(2) - 128)]),
    # adapters
    (lora, SHAPE, [dict(L=0), dict(R=0), dict(R=12), dict(R=264), dict(N=24), dict(N=0),
                   dict(K=48), dict(K=0), dict(M=0), dict(M=4000001), dict(ldx=64), dict(ldb=56),
                   dict(ldy=56), dict(ldx=1 << 28), dict(ldy=1 << 28), dict(K=32 * (1 << 40)),
                   dict(N=16 * (1 << 40)), dict(R=8, N=16776976, ldb=16776976, ldy=16776976),
                   dict(R=8, K=(1 << 26) + 32, ldx=(1 << 26) + 32)]),
    (lora, NULL, [dict(a=None), dict(b=None), dict(x=None), dict(ids=None), dict(base=None),
                  dict(y=None)]),
    (lora, ALIGN, [dict(a=A(0) + 8), dict(b=A(1) + 2), dict(x=A(3) + 8), dict(ldx=100),
                   dict(ids=A(4) + 2), dict(base=A(5) + 8), dict(ldb=68), dict(y=A(6) + 8),
                   dict(ldy=68), dict(s=A(2) + 2), dict(ws=A(7) + 8)]),
    (lora, WS, [dict(ws=None), dict(wsb=16)]),
    (lora, UNSUP, [dict(y=A(5) + 128), dict(y=A(5), ldy=128), dict(y=A(3)), dict(y=A(0)),
                   dict(y=A(4)), dict(ws=A(5)), dict(ws=A(6)), dict(ws=A(1)), dict(ws=A(2))]),
]
# calls that are in order: refused only for want of a device
VALID = [
    (norm, [dict(), dict(act=0), dict(act=0, xq=None, xc=None), dict(act=2),
            dict(act=2, ldq=0, ldc=0),
            dict(res=None, ldr=0), dict(sum=None, lds=0), dict(y=None, ldy=0), dict(sum=A(0)),
            dict(sum=A(1)), dict(sum=A(1), y=A(0)), dict(xc=A(6) + 1), dict(eps=0.0),
            dict(K=65536, ldx=65536, ldr=65536, lds=65536, ldy=65536, ldq=65536, ldc=2048),
            dict(M=4000000)]),
    (sort, [dict(), dict(T=5000, ws=A(4), wsb=1 << 20), dict(E=1024, T=3906, topk=1024, ws=A(4),
                                                             wsb=1 << 30)]),
    (grouped, [dict(), dict(elem=1), dict(layout=1), dict(epi=1, ldy=32), dict(rows=None),
               dict(x=None, xq=A(3), xc=A(7) + 1, ldq=256, ldc=8),
               dict(act=2, x=None, rows=None, xq=A(3), xc=A(7), ws=None, wsb=0, xrows=0, ldx=0),
               dict(xrows=4000000)]),
    (combine, [dict(), dict(T=1, topk=1, N=8), dict(ldys=72, ldy=80)]),
    (lora, [dict(), dict(s=None), dict(y=A(5)), dict(R=256, wsb=1 << 24), dict(ids=A(4) + 4)]),
]


@pytest.mark.parametrize("call,status,cases", REFUSED,
                         ids=[f"{c.__name__}-{s}" for c, s, _ in REFUSED])
def test_refusals(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_grouped_outputs_on_the_weights_are_refused():
    """y or the workspace anywhere in the packed weights or codes."""
    for elem, layout in ((0, 0), (0, 1), (1, 0)):
        wb, cb = mx.mx_packed_sizes(elem, layout, 4, 64, 256)
        last_w, last_c = (wb - 1) // 16 * 16, (cb - 1) // 16 * 16
        for kw in (dict(y=A(0)), dict(y=A(0) + last_w), dict(y=A(1)), dict(y=A(1) + last_c),
                   dict(y=A(0) - 2048), dict(ws=A(0) + 256), dict(ws=A(1) + last_c)):
            assert grouped(elem=elem, layout=layout, **kw) == UNSUP, (elem, layout, kw)


def test_grouped_outputs_behind_the_weights_are_in_order():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    for elem, layout in ((0, 0), (0, 1), (1, 0)):
        wb, cb = mx.mx_packed_sizes(elem, layout, 4, 64, 256)
        for kw in (dict(y=A(0) + (wb + 15) // 16 * 16), dict(ws=A(1) + (cb + 15) // 16 * 16)):
            assert grouped(elem=elem, layout=layout, **kw) == DEVICE, (elem, layout, kw)


def test_valid_calls_reach_the_device_gate():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    for call, cases in VALID:
        for kw in cases:
            assert call(**kw) == DEVICE, (call.__name__, kw)


def test_workspaces():
    L, b = mx.lib(), C.c_size_t()
    assert mx.mx_moe_sort_workspace(8, 256, 8) == 0
    assert mx.mx_moe_sort_workspace(8, 257, 8) > 0
    # the staged T16 activation, prequantized or not; nothing for T16 input
    for M, K in ((1, 32), (17, 160), (300, 1568)):
        qb, cb = mx.mx_act_t16_sizes(M, K)
        for given in (0, 1):
            need = mx.mx_grouped_workspace(0, 0, 4, 64, K, M, 1, given)
            assert need == (qb + 255) // 256 * 256 + cb
        assert mx.mx_grouped_workspace(1, 0, 4, 64, K, M, 2, 1) == 0
    # at least one fp32 partial product per row and rank, ranks padded to 16
    for M, R, K in ((1, 8, 32), (16, 16, 7168), (4096, 72, 7168)):
        assert mx.mx_lora_workspace(4, R, 64, K, M) >= M * ((R + 15) // 16 * 16) * 4
    assert L.mx_moe_sort_workspace(8, 4, 2, None) == NULL
    assert L.mx_grouped_workspace(0, 0, 4, 64, 256, 20, 1, 0, None) == NULL
    assert L.mx_lora_workspace(3, 16, 64, 96, 5, None) == NULL
    assert L.mx_grouped_workspace(0, 0, 4, 64, 256, 20, 0, 0, C.byref(b)) == UNSUP


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4096, dtype=torch.int16)
    i = torch.zeros(64, dtype=torch.int32)
    for call in (
            lambda: mx.mx_add_rms_norm(1, 32, t, 32, None, 0, t, 1e-6, 0, 0, None, 0, t, 32, None,
                                       0, None, 0, stream=0),
            lambda: mx.mx_moe_sort(8, 4, 2, i, i, i, i, None, 0, stream=0),
            lambda: mx.mx_moe_combine(1, 1, 8, 1, A(0), 8, A(1), A(2), t, 8, stream=0),
            lambda: mx.mx_grouped_linear(0, 0, 1, 16, 32, A(0), A(1), 1, i, 1, 0, 1, A(2), 32, None,
                                         0, None, 0, None, 0, A(3), 16, A(4), 1 << 20, stream=0),
            lambda: mx.mx_lora_add(1, 8, 16, 32, A(0), A(1), None, 1, t, 32, A(2), A(3), 16, A(3),
                                   16, A(4), 1 << 20, stream=0)):
        with pytest.raises(ValueError, match="not on the current GPU"):
            call()
    with pytest.raises(mx.MXError, match="mx_moe_sort"):
        mx.mx_moe_sort(0, 4, 2, A(0), A(1), A(2), A(3), None, 0, stream=0)


def test_host_code_under_sanitizers(tmp_path):
    """Every call above on a build of the host code under both sanitizers, with
    a fake gfx950 device and launchers that only count."""
    from test_sanitizers import CSRC, _asan_runtime, _env
    asan = _asan_runtime()
    lib = str(tmp_path / "libmx_ops_san.so")
    src = [os.path.join(CSRC, f) for f in ("mx_api.cpp", "mx_ops_api.cpp", "mx_plan.cpp")]
    src += [os.path.join(ROOT, "tests", "sanitize", f) for f in ("host_stubs.cpp", "ops_stubs.cpp")]
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-fno-omit-frame-pointer", *src, "-o", lib], capture_output=True, text=True)
    if r.returncode != 0 and "hip_runtime.h" in r.stderr:
        pytest.skip("HIP headers not found")
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True,
                       text=True, env=_env(asan, MX_LOG="1"), timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "operators' host checks ok" in r.stdout
    for name in ("add_rms_norm_kernel", "moe_place_kernel", "stage_rows_kernel", "grouped:",
                 "moe_gather_sum_kernel", "lora_expand_kernel"):
        assert name in r.stderr, f"no trace line for {name}"


def _checks(path):
    """In the child process: the host build in place of the library."""
    mx.LIB_PATH = path
    launches = C.c_long.in_dll(mx.lib(), "mx_ops_launches")
    for call, status, cases in REFUSED:
        for kw in cases:
            got = call(**kw)
            assert got == status, (call.__name__, kw, got)
    assert launches.value == 0, "a refused call launched"
    for call, cases in VALID:
        for kw in cases:
            before = launches.value
            got = call(**kw)
            assert got == OK, (call.__name__, kw, got)
            assert launches.value > before
    print("operators' host checks ok", launches.value)


if __name__ == "__main__":
    _checks(sys.argv[1])
