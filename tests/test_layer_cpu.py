"""CPU-side tests of the operators between a layer's products: every refusal that
the header names comes before any device work, with the documented status; the
binding refuses tensors that are not on the current GPU; the same calls run under
AddressSanitizer and UndefinedBehaviorSanitizer on a host-only build; the 64-bit
definitions that the GPU tests use, against differences and hand-made values."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import microscaling_quantized_linear_amd as mx  # noqa: E402

OK, NULL, SHAPE, ALIGN, VALUE, UNSUP, DEVICE, WS, LAUNCH = range(9)
BIG = 2 ** 62
INF, NAN = float("inf"), float("nan")


def A(i):
    """Fake, distinct, 256-byte aligned device addresses, 1 TiB apart: never dereferenced."""
    return (i + 1) << 40


def route(**kw):
    a = dict(E=64, T=5, topk=4, type=1, x=A(0), ldx=64, score=1, bias=A(1), groups=8, keep=4, best=2,
             renorm=1, scale=2.5, ids=A(2), w=A(3))
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_moe_route(*a.values(), None)


def block(**kw):
    a = dict(M=4, K=64, x=A(0), ldx=64, post=A(1), gate=A(2), gates=3, ldg=64, gid=A(3), type=0,
             res=A(4), ldr=64, alpha=1.0, w=A(5), offset=0.0, eps=1e-6, act=1, rule=0, sum=A(6),
             lds=64, y=A(7), ldy=64, xq=A(8), ldq=64, xc=A(9), ldc=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_block_norm(*a.values(), None)


def linear(**kw):
    a = dict(elem=0, layout=0, N=64, K=256, w=A(0), c=A(1), M=20, act=1, rule=0, x=A(2), ldx=256,
             xq=None, ldq=0, xc=None, ldc=0, bias=A(3), fn=3, gated=0, res=A(4), ldr=64, y=A(5),
             ldy=64, ws=A(6), wsb=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return mx.lib().mx_linear_epilogue(*a.values(), None)


GIVEN = dict(x=None, xq=A(2), ldq=256, xc=A(7), ldc=8)
T16 = dict(act=2, x=None, xq=A(2), xc=A(7))
REFUSED = [
    # routing
    (route, SHAPE, [dict(E=0), dict(E=1032, ldx=1032), dict(T=0), dict(T=-1), dict(topk=0),
                    dict(topk=65, ldx=64), dict(E=256, ldx=256, topk=65, keep=8),
                    dict(T=1000001), dict(T=BIG), dict(ldx=63), dict(ldx=BIG), dict(groups=0),
                    dict(groups=7), dict(E=130, ldx=130, groups=65, keep=65), dict(keep=0),
                    dict(keep=9), dict(topk=33), dict(groups=64, keep=3, best=1), dict(groups=64, best=2), dict(scale=NAN),
                    dict(scale=INF), dict(groups=-8), dict(keep=-1)]),
    (route, NULL, [dict(x=None), dict(ids=None), dict(w=None)]),
    (route, ALIGN, [dict(x=A(0) + 2), dict(type=0, x=A(0) + 1), dict(bias=A(1) + 2),
                    dict(ids=A(2) + 2), dict(w=A(3) + 1)]),
    (route, UNSUP, [dict(type=2), dict(score=2), dict(best=3), dict(best=0), dict(renorm=2),
                    dict(bias=None), dict(ids=A(0)), dict(w=A(0) + 64), dict(ids=A(1)), dict(w=A(1)),
                    dict(w=A(2)), dict(w=A(2) + 76)]),
    # the norms around a block
    (block, SHAPE, [dict(M=0), dict(M=4000001), dict(K=48), dict(K=0), dict(K=65568, ldx=65568),
                    dict(ldx=32), dict(ldr=56), dict(lds=32), dict(ldy=32), dict(ldq=48),
                    dict(ldc=1), dict(eps=-1e-6), dict(eps=NAN), dict(alpha=NAN), dict(alpha=INF),
                    dict(offset=-INF), dict(gates=0), dict(gates=4000001), dict(ldg=56),
                    dict(ldx=BIG), dict(ldg=BIG), dict(ldr=BIG), dict(M=-1), dict(K=-64)]),
    (block, NULL, [dict(x=None), dict(xq=None), dict(xc=None), dict(act=0, y=None),
                   dict(act=2, xc=None), dict(w=None, act=0, sum=None, y=None)]),
    (block, ALIGN, [dict(x=A(0) + 8), dict(ldx=68), dict(post=A(1) + 2), dict(gate=A(2) + 8),
                    dict(ldg=68), dict(gid=A(3) + 2), dict(res=A(4) + 2), dict(ldr=68),
                    dict(type=1, ldr=66), dict(w=A(5) + 2), dict(sum=A(6) + 8), dict(lds=68),
                    dict(type=1, lds=66), dict(y=A(7) + 4), dict(ldy=68), dict(xq=A(8) + 8),
                    dict(ldq=72), dict(act=2, xc=A(9) + 4)]),
    (block, UNSUP, [dict(act=3), dict(rule=2), dict(act=0, rule=5), dict(type=2),
                    dict(w=None), dict(w=None, act=0),                   # y without its norm
                    dict(sum=A(0) + 16), dict(sum=A(0), lds=128), dict(sum=A(4) + 128),
                    dict(y=A(6)), dict(y=A(1)), dict(sum=A(1)), dict(sum=A(2)), dict(sum=A(3)),
                    dict(sum=A(5)), dict(y=A(2)), dict(y=A(3)), dict(y=A(5)), dict(xq=A(0)),
                    dict(xq=A(4)), dict(xq=A(6)), dict(xq=A(7)), dict(xc=A(7)), dict(xc=A(8)),
                    dict(xq=A(2) + 256), dict(sum=A(0), y=A(0)), dict(act=2, xq=A(5)),
                    dict(act=2, xc=A(8) + 1024),
                    # an fp32 stream does not stand on bf16 rows
                    dict(type=1, sum=A(0)), dict(type=1, y=A(4))]),
    # the linear with an epilogue
    (linear, SHAPE, [dict(N=40), dict(N=0), dict(K=100), dict(K=0), dict(M=0), dict(ldx=128),
                     dict(ldy=56), dict(ldr=56), dict(gated=1, ldy=24), dict(gated=1, ldr=24),
                     dict(M=BIG), dict(ldx=BIG), dict(ldy=BIG), dict(ldr=BIG), dict(N=16 * (1 << 40)),
                     dict(K=32 * (1 << 40)), dict(N=1 << 24, K=128, ldx=128, ldy=1 << 24, ldr=1 << 24),
                     dict(M=20, ldr=1 << 26), dict(M=20, ldy=1 << 26),
                     dict(act=0, M=1048561, K=32, ldx=32), dict(GIVEN, ldq=240),
                     dict(GIVEN, ldc=7), dict(GIVEN, ldq=BIG), dict(GIVEN, ldc=BIG),
                     dict(layout=1, N=48)]),
    (linear, NULL, [dict(w=None), dict(c=None), dict(y=None), dict(x=None), dict(T16, xq=None),
                    dict(T16, xc=None)]),
    (linear, ALIGN, [dict(w=A(0) + 8), dict(c=A(1) + 4), dict(y=A(5) + 8), dict(ldy=68),
                     dict(x=A(2) + 2), dict(ldx=260), dict(bias=A(3) + 1), dict(res=A(4) + 8),
                     dict(ldr=68), dict(ws=A(6) + 8), dict(GIVEN, xq=A(2) + 8), dict(GIVEN, ldq=264),
                     dict(T16, xc=A(7) + 4)]),
    (linear, UNSUP, [dict(elem=2), dict(layout=2), dict(elem=1), dict(act=3), dict(rule=2),
                     dict(fn=6), dict(fn=-1), dict(gated=2), dict(gated=-1),
                     dict(elem=1, layout=1, act=0),
                     dict(y=A(0)), dict(y=A(1)), dict(y=A(2)), dict(y=A(3) - 128), dict(y=A(4) + 128),
                     dict(y=A(4), ldy=128), dict(ws=A(0)), dict(ws=A(2)), dict(ws=A(3)), dict(ws=A(4)),
                     dict(ws=A(5)), dict(GIVEN, y=A(2)), dict(GIVEN, y=A(7)), dict(T16, y=A(2)),
                     dict(T16, y=A(7))]),
    (linear, WS, [dict(ws=None), dict(wsb=100)]),
]
# calls that are in order: refused only for want of a device
VALID = [
    (route, [dict(), dict(bias=None, best=1), dict(type=0, x=A(0) + 2), dict(groups=1, keep=1, best=1),
             dict(score=0, renorm=0), dict(E=1024, ldx=1030, groups=64, keep=64, topk=64, T=62500),
             dict(E=1, ldx=1, groups=1, keep=1, topk=1, T=4000000, best=1),
             dict(x=A(0) + 4), dict(groups=64, keep=4, best=1), dict(groups=32, keep=4, best=2), dict(scale=-1.0)]),
    (block, [dict(), dict(act=0), dict(act=0, xq=None, xc=None), dict(act=2), dict(act=2, ldq=0, ldc=0),
             dict(res=None, ldr=0), dict(sum=None, lds=0), dict(y=None, ldy=0), dict(sum=A(0)),
             dict(sum=A(4)), dict(sum=A(4), y=A(0)), dict(sum=A(0), y=A(4)), dict(xc=A(9) + 1),
             dict(eps=0.0), dict(post=None), dict(gate=None, gates=0, ldg=0), dict(gid=None),
             dict(gate=None, gid=A(3) + 1), dict(w=None, act=0, y=None), dict(type=1),
             dict(type=1, ldr=68, lds=68), dict(type=1, sum=A(4)), dict(type=1, y=A(0)),
             dict(w=None, act=0, y=None, type=1, sum=A(4)), dict(M=4000000), dict(offset=1.0),
             dict(K=65536, ldx=65536, ldr=65536, lds=65536, ldy=65536, ldq=65536, ldc=2048,
                  ldg=65536)]),
    (linear, [dict(), dict(gated=1, ldy=32, ldr=32), dict(res=None, ldr=0), dict(bias=None),
              dict(fn=0, res=None, ldr=0), dict(y=A(4)), dict(act=0, ws=None, wsb=0),
              dict(elem=1, act=0, ws=None, wsb=0), dict(layout=1), dict(GIVEN, ws=None, wsb=0),
              dict(T16, ws=None, wsb=0), dict(M=300, wsb=1 << 24), dict(bias=A(3) + 2),
              dict(GIVEN, M=300, wsb=1 << 24)] + [dict(fn=f) for f in range(6)]),
]


@pytest.mark.parametrize("call,status,cases", REFUSED,
                         ids=[f"{c.__name__}-{s}" for c, s, _ in REFUSED])
def test_refusals(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_valid_calls_reach_the_device_gate():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    for call, cases in VALID:
        for kw in cases:
            assert call(**kw) == DEVICE, (call.__name__, kw)


def test_linear_outputs_on_the_weights_are_refused():
    """y or the workspace anywhere in the packed weights or codes."""
    for elem, layout, act in ((0, 0, 1), (0, 1, 1), (1, 0, 0)):
        wb, cb = mx.mx_packed_sizes(elem, layout, 1, 64, 256)
        last_w, last_c = (wb - 1) // 16 * 16, (cb - 1) // 16 * 16
        for kw in (dict(y=A(0) + last_w), dict(y=A(1) + last_c), dict(y=A(0) - 2048)):
            assert linear(elem=elem, layout=layout, act=act, **kw) == UNSUP, (elem, layout, kw)
        if act:
            assert linear(elem=elem, layout=layout, ws=A(1) + last_c) == UNSUP


def test_columns_of_one_buffer_are_apart():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    at = lambda c, size=2: A(20) + c * size                                     # noqa: E731
    assert block(x=at(0), ldx=256, sum=at(64), lds=256, y=at(128), ldy=256, res=at(192),
                 ldr=256) == DEVICE
    assert block(x=at(0), ldx=256, sum=at(56), lds=256) == UNSUP
    assert linear(res=at(64), ldr=128, y=at(0), ldy=128) == DEVICE
    assert linear(res=at(64), ldr=128, y=at(8), ldy=128) == UNSUP
    assert linear(x=at(0), ldx=512, y=at(256), ldy=512) == DEVICE


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4096, dtype=torch.int16)
    for call in (
            lambda: mx.mx_moe_route(8, 1, 2, 1, t, 8, 0, None, 1, 1, 1, True, 1.0, A(0), A(1), stream=0),
            lambda: mx.mx_block_norm(1, 32, A(0), 32, None, None, 0, 0, None, 0, t, 32, 1.0, A(1), 0.0,
                                     1e-6, 0, 0, None, 0, A(2), 32, None, 0, None, 0, stream=0),
            lambda: mx.mx_linear_epilogue(0, 0, 16, 32, A(0), A(1), 1, 0, 0, A(2), 32, None, 0, None, 0,
                                          None, 3, False, t, 16, A(3), 16, None, 0, stream=0)):
        with pytest.raises(ValueError, match="not on the current GPU"):
            call()
    with pytest.raises(mx.MXError, match="mx_moe_route"):
        mx.mx_moe_route(0, 1, 2, 1, A(0), 8, 0, None, 1, 1, 1, True, 1.0, A(1), A(2), stream=0)


@pytest.fixture(params=["compiled", "ctypes"])
def path(request, monkeypatch):
    """Either way from Python to the entry points."""
    if request.param == "compiled":
        assert mx._mxcall is not None, "_mxcall is not built"
    else:
        monkeypatch.setattr(mx, "_mxcall", None)
    monkeypatch.setattr(mx.lib(), "direct", {})
    return request.param


def test_either_call_path_refuses_the_same(path):
    for call, status, cases in REFUSED:
        for kw in cases:
            assert call(**kw) == status, (path, call.__name__, kw)


def test_either_call_path_takes_the_same_arguments(path):
    import torch
    t = torch.zeros(4096, dtype=torch.int16)
    args = dict(E=8, T=1, topk=9, type=1, logits=A(0), ldl=8, score=0, bias=None, groups=1, topk_groups=1,
                group_best=1, renorm=True, scale=1, topk_ids=A(1), topk_weights=A(2), stream=0)

    def run(**kw):
        return mx.mx_moe_route(**dict(args, **kw))

    class Stream:
        cuda_stream = 1 << 40
    for kw in (dict(), dict(renorm=np.bool_(True)), dict(scale=np.float64(2.0)), dict(stream=Stream()),
               dict(topk=True, E=0), dict(logits=2 ** 64 - 256)):
        with pytest.raises(mx.MXError):               # topk or E: refused behind the marshalling
            run(**kw)
    with pytest.raises(ValueError, match="on cpu, not on the current GPU"):
        run(topk_weights=t)
    # what is no number, address, tensor or stream
    for kw in (dict(E="8"), dict(topk=2.5), dict(scale="1"), dict(scale=None), dict(ldl=None)):
        with pytest.raises((TypeError, C.ArgumentError)):
            run(**kw)
    for kw in (dict(bias="x"), dict(stream="x")):
        with pytest.raises(AttributeError):
            run(**kw)


# ---- the definitions ---------------------------------------------------------------------


def test_route_definition():
    import layer_ref as ref
    x = np.array([[1.0, 3.0, 3.0, -1.0], [-INF, NAN, -INF, -INF], [INF, 2.0, NAN, INF]])
    ids, w, _ = ref.route(x, ref.SOFTMAX, None, 1, 1, 1, 2, True, 1.0)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 3]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [0.5, 0.5]])
    # the bias orders and does not weigh
    b = np.array([0.0, -1.0, 0.0, 0.9], np.float32)
    ids, w, _ = ref.route(x[:1], ref.SIGMOID, b, 1, 1, 1, 3, False, 2.0)
    assert ids.tolist() == [[3, 2, 0]]
    assert np.allclose(w, 2 / (1 + np.exp([[1.0, -3.0, -1.0]])))
    # two groups of two: the sum of two against the largest
    x = np.array([[4.0, -4.0, 1.0, 1.5]])
    z = np.zeros(4, np.float32)
    assert ref.route(x, ref.SIGMOID, z, 2, 1, 2, 2, True, 1.0)[0].tolist() == [[3, 2]]
    assert ref.route(x, ref.SIGMOID, None, 2, 1, 1, 2, True, 1.0)[0].tolist() == [[0, 1]]


def test_epilogue_definition():
    """The activations' slopes that the bounds use, against differences; known values."""
    import layer_ref as ref
    z = np.linspace(-12, 12, 4801)
    h = 1e-5
    for kind in range(6):
        slope = (ref.fn(kind, z + h) - ref.fn(kind, z - h)) / (2 * h)
        assert (np.abs(slope) <= ref._slope(kind, z, h) + 1e-6).all(), kind
    assert np.allclose(ref.fn(ref.GELU, np.array([-1.0, 0.0, 1.0])), [-0.158655254, 0, 0.841344746])
    assert np.allclose(ref.fn(ref.SILU, np.array([2.0])), [1.761594156])
    assert np.abs(ref.fn(ref.GELU_TANH, z) - ref.fn(ref.GELU, z)).max() < 1e-3


def test_host_code_under_sanitizers(tmp_path):
    """Every call above on a build of the host code under both sanitizers, with a
    fake gfx950 device and launchers that only count."""
    from test_sanitizers import CSRC, _asan_runtime, _env
    asan = _asan_runtime()
    lib = str(tmp_path / "libmx_layer_san.so")
    src = [os.path.join(CSRC, f) for f in ("mx_api.cpp", "mx_layer_api.cpp", "mx_plan.cpp")]
    src += [os.path.join(ROOT, "tests", "sanitize", f) for f in ("host_stubs.cpp", "layer_stubs.cpp")]
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
    assert "layer host checks ok" in r.stdout
    for name in ("route_kernel", "block_norm_kernel", "with epilogue"):
        assert name in r.stderr, f"no trace line for {name}"


def _checks(path):
    """In the child process: the host build in place of the library."""
    mx.LIB_PATH = path
    counts = [C.c_long.in_dll(mx.lib(), n) for n in ("mx_layer_launches", "mx_stub_launches")]
    launches = lambda: sum(c.value for c in counts)                             # noqa: E731
    for call, status, cases in REFUSED:
        for kw in cases:
            got = call(**kw)
            assert got == status, (call.__name__, kw, got)
    assert launches() == 0, "a refused call launched"
    for call, cases in VALID:
        for kw in cases:
            before = launches()
            got = call(**kw)
            assert got == OK, (call.__name__, kw, got)
            assert launches() > before
    print("layer host checks ok", launches())


if __name__ == "__main__":
    _checks(sys.argv[1])
