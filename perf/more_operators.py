"""Measured cases of a decoder layer's operators between its quantized products.

Three operators that a serving program runs around ``mx_linear`` and the
routed experts:

* ``moe_route``        scores of router logits, a bias for balance, groups,
                       top-k, renormalised weights
* ``block_norm``       the norm after a block, its gate and the scaled residual
                       stream, the norm before the next block, MXFP8 output
* ``linear_epilogue``  the block-scaled product with bias, activation (gated or
                       not) and residual in its epilogue

A case is a dict of plain values.  ``prepare`` makes what the program holds
before the call (activations, packed weights, logits, output buffers) on the
GPU, from the seed alone; ``run`` is one call.  With ``own`` false, ``run``
computes the operator in elementary torch operations in 32 bits (the scores
that a bias orders in 64, as equal 32-bit scores tie); with ``own`` true it
calls the library.  ``exact`` computes it in 64 bits.

What is held in 8 bits comes back as torch's 8-bit floating types: e4m3 values
and E8M0 scales, in the layout that the call fills.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3, E2M1 = 0, 1
ROW32, BLK32 = 0, 1
OCP, CEIL448 = 0, 1
BF16, MXFP8, T16 = 0, 1, 2
FLOAT_BF16, FLOAT_F32 = 0, 1
SOFTMAX, SIGMOID = 0, 1
FN = dict(none=0, relu=1, relu2=2, silu=3, gelu=4, gelu_tanh=5)
EPS = 1e-6


def listed():
    return [
        # decode: 16 tokens over 32 experts, softmax weights over the chosen
        # (latency)
        dict(name="route_decode", op="route", E=32, T=16, topk=8, bf16=False, score=SOFTMAX,
             bias=False, groups=1, keep=1, best=1, renorm=True, pad=0.0),
        # prefill: sigmoid scores with a balance bias, four of eight groups
        dict(name="route_prefill_groups", op="route", E=256, T=16384, topk=8, bf16=False,
             score=SIGMOID, bias=True, groups=8, keep=4, best=2, renorm=True, pad=0.05),
        # an odd batch: bf16 logits (many ties), softmax over all experts,
        # padding tokens whose logits are all masked
        dict(name="route_ragged_bf16", op="route", E=128, T=4099, topk=6, bf16=True,
             score=SOFTMAX, bias=False, groups=1, keep=1, best=1, renorm=False, pad=0.1),
        # decode: both norms and a layer scale around a few tokens, fed to the
        # matrix cores' tile layout (latency)
        dict(name="block_norm_decode_t16", op="norm", M=4, K=7168, post=True, gates=1,
             stream=FLOAT_BF16, alpha=1.0, offset=0.0, act=T16, rule=OCP, keep=False),
        # prefill: an fp32 residual stream, one gate a sequence, weights stored
        # around zero, row-major bytes and the bf16 rows that the router reads
        dict(name="block_norm_prefill_f32", op="norm", M=4096, K=7168, post=True, gates=8,
             stream=FLOAT_F32, alpha=0.8, offset=1.0, act=MXFP8, rule=OCP, keep=True),
        # an odd batch with short rows, a bf16 stream, no quantized output
        dict(name="block_norm_ragged", op="norm", M=5001, K=1568, post=True, gates=0,
             stream=FLOAT_BF16, alpha=1.0, offset=0.0, act=BF16, rule=OCP, keep=True),
        # decode: gate and up products of a dense block, quantized in the call
        # (the weights' stream)
        dict(name="linear_decode_gate_up", op="linear", elem=E4M3, layout=BLK32, M=16, N=14336,
             K=7168, act=MXFP8, rule=OCP, bias=False, fn="silu", gated=True, residual=False),
        # decode: a projection back onto the residual stream, e2m1 weights
        dict(name="linear_decode_w4_residual", op="linear", elem=E2M1, layout=ROW32, M=4, N=4096,
             K=4096, act=BF16, rule=OCP, bias=True, fn="none", gated=False, residual=True),
        # the smallest rows of odd sizes: bf16 activations, a squared ReLU
        dict(name="linear_small_relu2", op="linear", elem=E4M3, layout=ROW32, M=8, N=4096, K=1568,
             act=BF16, rule=OCP, bias=True, fn="relu2", gated=False, residual=False),
        # a prompt's gate and up products, quantized by the norm ahead of it
        dict(name="linear_prefill_gate_up", op="linear", elem=E4M3, layout=BLK32, M=4096, N=7168,
             K=7168, act=T16, rule=OCP, bias=False, fn="silu", gated=True, residual=False),
        # its projection back onto the residual stream
        dict(name="linear_prefill_residual", op="linear", elem=E4M3, layout=ROW32, M=4096, N=7168,
             K=4096, act=MXFP8, rule=OCP, bias=False, fn="none", gated=False, residual=True),
        # a ragged batch through a biased GELU onto the residual
        dict(name="linear_ragged_gelu", op="linear", elem=E4M3, layout=BLK32, M=1001, N=4096,
             K=1568, act=MXFP8, rule=CEIL448, bias=True, fn="gelu", gated=False, residual=True),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear", "linear"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _between(rng, 4, 512 // groups)
        bias = rng.random() < 0.5
        keep = rng.randint(1, groups)
        return dict(op=op, E=E, T=_between(rng, 1, 8000), topk=rng.randint(1, min(10, E // groups * keep)),
                    bf16=rng.random() < 0.3, score=rng.choice([SOFTMAX, SIGMOID]), bias=bias,
                    groups=groups, keep=keep, best=rng.choice([1, 2]) if bias else 1,
                    renorm=rng.random() < 0.7, pad=rng.choice([0.0, 0.1]))
    if op == "norm":
        return dict(op=op, M=_between(rng, 1, 4000), K=32 * _between(rng, 1, 224),
                    post=rng.random() < 0.8, gates=rng.choice([0, 1, rng.randint(2, 64)]),
                    stream=rng.choice([FLOAT_BF16, FLOAT_F32]), alpha=rng.choice([1.0, 0.5, 1.25]),
                    offset=rng.choice([0.0, 1.0]), act=rng.choice([BF16, MXFP8, T16]),
                    rule=rng.choice([OCP, CEIL448]), keep=rng.random() < 0.5)
    elem = rng.choice([E4M3, E4M3, E4M3, E2M1])
    act = BF16 if elem == E2M1 else rng.choice([BF16, MXFP8, MXFP8, T16])
    # bf16 activations are the decode form
    M = _between(rng, 1, 64) if act == BF16 else _between(rng, 1, 4000)
    return dict(op=op, elem=elem, layout=rng.choice([ROW32, BLK32]) if elem == E4M3 else ROW32,
                M=M, N=32 * _between(rng, 1, 220), K=32 * _between(rng, 1, 220), act=act,
                rule=rng.choice([OCP, CEIL448]), bias=rng.random() < 0.5,
                fn=rng.choice(sorted(FN)), gated=rng.random() < 0.5, residual=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


class _Inputs:
    """Seeded tensors on the device."""

    def __init__(self, seed):
        self.device = _device()
        self.g = torch.Generator(self.device).manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=self.device)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device=self.device)

    def weight(self, elem, layout, N, K):
        """A normal weight in the elements' format, scaled to the fan-in:
        standard bytes [N, K or K/2] and codes [N, K/32] or [N/32, K/32]."""
        w = self.normal(N, K // 32, 32).mul_(K ** -0.5)
        amax = w.abs().amax(-1)                                     # [N, K/32]
        if layout == BLK32:
            amax = amax.view(N // 32, 32, K // 32).amax(1)
        code = ((amax.contiguous().view(torch.int32) >> 23) - (8 if elem == E4M3 else 2)).clamp_(0, 254)
        row = code if layout == ROW32 else code.repeat_interleave(32, dim=0)
        w.mul_(((254 - row) << 23).to(torch.int32).view(torch.float32).unsqueeze(-1))
        code = code.to(torch.uint8)
        if elem == E4M3:
            return w.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(N, K), code
        edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=self.device)
        nib = torch.bucketize(w.abs(), edge, out_int32=True).to(torch.uint8)
        nib += (w < 0).to(torch.uint8) * 8
        nib = nib.view(N, K // 2, 2)
        return nib[..., 0] | nib[..., 1] << 4, code


def _pack(elem, layout, N, K, w, codes):
    """The packed weight and codes that the library documents (what its load-time
    pack writes): 16-row tiles of 16-byte pieces; code dwords of four steps, a
    trailer with the smallest and largest code."""
    rowb = K if elem == E4M3 else K // 2
    wp = w.view(N // 16, 16, rowb // 16, 16).transpose(1, 2).contiguous().view(-1)
    Q = -(-K // 512)
    c = torch.full((codes.shape[0], 16 * Q), 128, dtype=torch.uint8, device=w.device)
    c[:, :K // 32] = codes
    if layout == ROW32:
        c = c.view(N // 16, 16, Q, 4, 4).permute(0, 2, 4, 1, 3)
    else:
        c = c.view(-1, Q, 4, 4).permute(0, 1, 3, 2)
    tail = torch.zeros(16, dtype=torch.uint8, device=w.device)
    tail[0], tail[1] = codes.min(), codes.max()
    return wp, torch.cat([c.reshape(-1), tail])


def _route_state(c, i):
    T, E, k = c["T"], c["E"], c["topk"]
    logits = 1.5 * i.normal(T, E) + 0.7 * i.normal(E)
    logits.masked_fill_(i.uniform(T, 1) < c["pad"], -math.inf)
    return dict(logits=logits.bfloat16() if c["bf16"] else logits,
                bias=0.1 * i.normal(E) if c["bias"] else None,
                ids=torch.empty(T, k, dtype=torch.int32, device=i.device),
                weights=torch.empty(T, k, dtype=torch.float32, device=i.device))


def _norm_state(c, i):
    M, K = c["M"], c["K"]
    channel = torch.where(i.uniform(K) < 0.01, 20.0, 1.0)     # a residual stream's large channels
    f = torch.float32 if c["stream"] == FLOAT_F32 else torch.bfloat16
    vector = lambda: (1 - c["offset"] + 0.2 * i.normal(K)).bfloat16()  # noqa: E731
    s = dict(x=i.normal(M, K).bfloat16(), residual=(2 * i.normal(M, K) * channel).to(f),
             weight=vector(), post=vector() if c["post"] else None, gate=None, ids=None)
    if c["gates"]:
        s["gate"] = (0.5 + 0.3 * i.normal(c["gates"], K)).bfloat16()
    if c["gates"] > 1:                      # a batch's rows, sequence by sequence, in any order
        s["ids"] = (torch.arange(M, device=i.device) * c["gates"] // M).to(torch.int32)
        s["ids"] = s["ids"][torch.argsort(i.uniform(M))].contiguous()
    s["sum"] = torch.empty_like(s["residual"])
    s["y"] = torch.empty_like(s["x"]) if c["keep"] or c["act"] == BF16 else None
    if c["act"] != BF16:
        S = -(-K // 128)
        n, m = ((M * K, M * (K // 32)) if c["act"] == MXFP8 else
                (-(-M // 16) * S * 2048, -(-M // 16) * (-(-S // 4)) * 256))
        s["xq"] = torch.empty(n, dtype=torch.uint8, device=i.device)
        s["xcodes"] = torch.empty(m, dtype=torch.uint8, device=i.device)
    return s


def _linear_state(c, i):
    N, K, M = c["N"], c["K"], c["M"]
    w, codes = i.weight(c["elem"], c["layout"], N, K)
    s = dict(w=w, codes=codes)
    s["w_packed"], s["codes_packed"] = _pack(c["elem"], c["layout"], N, K, w, codes)
    x = i.normal(M, K)
    s["x"] = torch.where(i.uniform(M, K) < 0.01, 20 * x, x).bfloat16()
    if c["act"] == T16:                     # handed over by the norm ahead of the product
        q, code = _quantize(s["x"].float(), c["rule"])
        s["q"], s["code"] = q, code
        s["xq"], s["xcodes"] = _to_t16(q.view(torch.uint8), code, M, K)
    width = N // 2 if c["gated"] else N
    s["bias"] = i.normal(N).bfloat16() if c["bias"] else None
    s["residual"] = i.normal(M, width).mul_(2).bfloat16() if c["residual"] else None
    s["y"] = torch.empty(M, width, dtype=torch.bfloat16, device=i.device)
    return s


def prepare(case, seed):
    make = dict(route=_route_state, norm=_norm_state, linear=_linear_state)[case["op"]]
    return dict(make(case, _Inputs(seed)), case=case)


# ---- plain forms, 32 bits -------------------------------------------------------------


def _quantize(x, rule):
    """MXFP8 of fp32 rows holding bf16 values: e4m3 [M, K], E8M0 codes (uint8)
    [M, K/32]."""
    M, K = x.shape
    b = x.view(M, K // 32, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    code = (bits >> 23) - 8
    if rule == CEIL448:
        code = code + ((bits & 0x7FFFFF) > 0x600000).int()
    code = torch.where(bits >> 23 == 0, 0, code).clamp(0, 254)
    scale = ((254 - code) << 23).to(torch.int32).view(torch.float32)
    q = (b * scale.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(M, K), code.to(torch.uint8)


def _to_t16(v, c, M, K):
    """Values [M, K] and codes [M, K/32] in the 16-token tile layout."""
    S, MB = -(-K // 128), -(-M // 16)
    Q = -(-S // 4)
    d = torch.zeros(MB * 16, S * 128, dtype=v.dtype, device=v.device)
    d[:M, :K] = v
    e = torch.full((MB * 16, Q * 16), 127, dtype=c.dtype, device=c.device)
    e[:M, :K // 32] = c
    return (d.view(MB, 16, S, 2, 4, 16).permute(0, 2, 3, 4, 1, 5).reshape(-1),
            e.view(MB, 16, Q, 4, 4).permute(0, 2, 4, 1, 3).reshape(-1))


def _scores64(x, score):
    """Scores of 64-bit logits; a masked logit (-inf) scores 0."""
    if score == SIGMOID:
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True).clamp_min(-1e300))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def _route(s, c):
    T, E, k = c["T"], c["E"], c["topk"]
    x = s["logits"].float()
    score = _scores64(x.double(), c["score"]).float()
    # with a bias the order is that of the biased scores, else that of the logits
    key = torch.where(x == -math.inf, -math.inf, score + s["bias"]) if c["bias"] else x
    if c["groups"] > 1:
        best = key.view(T, c["groups"], -1).sort(2, descending=True)[0][..., :c["best"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device)
        kept.scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(E // c["groups"], 1), key, -math.inf)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    live = key[:, :k] > -math.inf
    w = torch.where(live, score.gather(1, ids[:, :k]), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    return [torch.where(live, ids[:, :k], -1).to(torch.int32), 2.5 * w]


def _norm(s, c):
    p = s["x"].float()
    if c["post"]:
        p = p * torch.rsqrt(p.square().mean(-1, keepdim=True) + EPS) * (c["offset"] + s["post"].float())
    if c["gates"]:
        g = s["gate"].float()
        p = p * (g[s["ids"].long()] if s["ids"] is not None else g)
    total = (c["alpha"] * s["residual"].float() + p).to(s["sum"].dtype)
    v = total.float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * (c["offset"] + s["weight"].float())
    y = y.bfloat16()
    out = [total, y if s["y"] is not None else None]
    if c["act"] == BF16:
        return out
    q, code = _quantize(y.float(), c["rule"])
    q = q.view(torch.uint8)
    if c["act"] == T16:
        q, code = _to_t16(q, code, c["M"], c["K"])
    return out + [q.reshape(-1).view(torch.float8_e4m3fn), code.reshape(-1).view(torch.float8_e8m0fnu)]


def _weight32(s, c):
    N, K = c["N"], c["K"]
    if c["elem"] == E4M3:
        w = s["w"].view(torch.float8_e4m3fn).float()
    else:
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                             device=s["w"].device)
        w = torch.stack([value[(s["w"] & 15).int()], value[(s["w"] >> 4).int()]], -1)
    scale = (s["codes"].int() << 23).view(torch.float32).view(-1, K // 32)
    if c["layout"] == BLK32:
        scale = scale.repeat_interleave(32, dim=0)
    return (w.view(N, K // 32, 32) * scale.unsqueeze(-1)).view(N, K)


def _function(z, fn):
    if fn == "relu":
        return z.clamp_min(0)
    if fn == "relu2":
        return z.clamp_min(0).square()
    if fn == "silu":
        return z / (1 + torch.exp(-z))
    if fn == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if fn == "gelu_tanh":                   # 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2 u))
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _linear(s, c):
    if c["act"] == BF16:
        a = s["x"].float()
    else:
        q, code = (s["q"], s["code"]) if c["act"] == T16 else _quantize(s["x"].float(), c["rule"])
        a = (q.float().view(-1, c["K"] // 32, 32) *
             (code.int() << 23).view(torch.float32).unsqueeze(-1)).view(-1, c["K"])
    z = torch.mm(a, _weight32(s, c).t())
    if c["bias"]:
        z = z + s["bias"].float()
    h = _function(z[:, 0::2], c["fn"]) * z[:, 1::2] if c["gated"] else _function(z, c["fn"])
    if c["residual"]:
        h = h + s["residual"].float()
    return h.bfloat16()


# ---- the library's calls --------------------------------------------------------------


def _own(s, c):
    import microscaling_quantized_linear_amd as mx

    op = c["op"]
    if op == "route":
        mx.mx_moe_route(c["E"], c["T"], c["topk"], FLOAT_BF16 if c["bf16"] else FLOAT_F32,
                        s["logits"], c["E"], c["score"], s["bias"], c["groups"], c["keep"],
                        c["best"], c["renorm"], 2.5, s["ids"], s["weights"])
        return [s["ids"], s["weights"]]
    M, K = c["M"], c["K"]
    if op == "norm":
        y = s["y"]
        mx.mx_block_norm(M, K, s["x"], K, s["post"], s["gate"], c["gates"], K, s["ids"],
                         c["stream"], s["residual"], K, c["alpha"], s["weight"], c["offset"], EPS,
                         c["act"], c["rule"], s["sum"], K, y, K if y is not None else 0,
                         s.get("xq"), K, s.get("xcodes"), K // 32)
        out = [s["sum"], y]
        if c["act"] == BF16:
            return out
        return out + [s["xq"].view(torch.float8_e4m3fn), s["xcodes"].view(torch.float8_e8m0fnu)]
    N, y = c["N"], s["y"]
    ws = s.get("ws")
    if ws is None:                         # kept by the program for its next calls
        need = mx.mx_linear_workspace(c["elem"], c["layout"], N, K, M, c["act"], c["act"] == T16)
        ws = s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=y.device)
    mx.mx_linear_epilogue(c["elem"], c["layout"], N, K, s["w_packed"], s["codes_packed"], M,
                          c["act"], c["rule"], None if c["act"] == T16 else s["x"], K,
                          s.get("xq"), 0, s.get("xcodes"), 0, s["bias"], FN[c["fn"]], c["gated"],
                          s["residual"], y.shape[1] if c["residual"] else 0, y, y.shape[1], ws,
                          ws.numel())
    return y


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return dict(route=_route, norm=_norm, linear=_linear)[c["op"]](state, c)


def work(case):
    """Each input read once, each output written once; the products' operations."""
    c = case
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return dict(bytes=n * (2 if c["bf16"] else 4) + 8 * c["T"] * c["topk"] + 4 * c["E"], flops=8 * n)
    M, K = c["M"], c["K"]
    if c["op"] == "norm":
        n = M * K
        per = 2 + (8 if c["stream"] == FLOAT_F32 else 4) + (2 if c["keep"] or c["act"] == BF16 else 0)
        rows = -(-M // 16) * 16 if c["act"] == T16 else M
        return dict(bytes=n * per + (0 if c["act"] == BF16 else rows * K * 33 / 32) +
                    2 * K * (1 + c["post"] + c["gates"]), flops=16 * n)
    N = c["N"]
    width = N // 2 if c["gated"] else N
    codes = N * K / 32 / (32 if c["layout"] == BLK32 else 1)
    x = M * K * (33 / 32 if c["act"] == T16 else 2)
    return dict(bytes=N * K * (1 if c["elem"] == E4M3 else 0.5) + codes + x +
                M * width * (4 if c["residual"] else 2) + (2 * N if c["bias"] else 0),
                flops=2 * M * N * K)


# ---- 64 bits --------------------------------------------------------------------------


def _pow2(code):
    return torch.exp2(code.double() - 127)


def _codes64(v, rule):
    """E8M0 codes of 64-bit blocks [..., 32]."""
    amax = v.abs().amax(-1)
    if rule == OCP:
        e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -140))) - 8
    else:
        e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -126) / 448))
    return torch.where(amax < 2.0 ** -126, torch.zeros_like(amax), (e + 127).clamp(0, 254))


def _round_to(v, bits, low):
    """64-bit values rounded once, to nearest even, to `bits` significant bits
    (fewer below 2^low)."""
    _, e = torch.frexp(v)
    step = torch.exp2(e.double().clamp_min(low) - bits)
    return torch.round(v / step) * step


def _e4m3_table(device):
    b = torch.arange(256, device=device)
    e, m = (b >> 3 & 15).double(), (b & 7).double()
    v = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(e - 6) * m / 8)
    return torch.where(b >= 128, -v, v)


def _e2m1_table(device):
    b = torch.arange(16, device=device)
    e, m = (b >> 1 & 3).double(), (b & 1).double()
    v = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)
    return torch.where(b >= 8, -v, v)


def _ahead(key):
    """[T, n]: how many of a row come ahead of each: the larger, and the equal of
    a lower index."""
    n = key.shape[1]
    a, b = key.unsqueeze(2), key.unsqueeze(1)
    lower = torch.arange(n, device=key.device)
    lower = lower.unsqueeze(0) < lower.unsqueeze(1)
    return ((b > a) | ((b == a) & lower)).sum(2)


def _exact_route(s, c):
    T, E, k, G = c["T"], c["E"], c["topk"], c["groups"]
    out = []
    for x in s["logits"].double().split(max(1, 2 ** 26 // (E * E))):
        if c["score"] == SIGMOID:
            p = torch.sigmoid(x)
        else:
            p = torch.softmax(x, 1).nan_to_num(0.0)
        masked = x == -math.inf
        if c["bias"]:
            key = (p.float() + s["bias"]).double().masked_fill(masked, -math.inf)
        else:
            key = x
        if G > 1:
            n = E // G
            by = key.view(-1, n)
            near = torch.where(_ahead(by) < c["best"], by, 0.0).sum(1).float().double().view(-1, G)
            gone = _ahead(near) >= c["keep"]
            key = key.masked_fill(gone.repeat_interleave(n, 1), -math.inf)
        place = _ahead(key)
        chosen = (place < k) & (key > -math.inf)
        w = torch.zeros(x.shape[0], E, dtype=torch.float64, device=x.device)
        w.scatter_(1, place, torch.where(chosen, p, 0.0))
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        out.append(2.5 * w[:, :k])
    return [None, torch.cat(out)]


def _exact_norm(s, c):
    M, K = c["M"], c["K"]
    p = s["x"].double()
    if c["post"]:
        p = p / torch.sqrt((p * p).sum(-1, keepdim=True) / K + EPS) * (s["post"].double() + c["offset"])
    if s["gate"] is not None:
        rows = torch.zeros(M, dtype=torch.long, device=p.device) if s["ids"] is None else s["ids"].long()
        p = p * s["gate"].double()[rows]
    total = s["residual"].double() * float(torch.tensor(c["alpha"], dtype=torch.float32)) + p
    v = _round_to(total, 24, -125) if c["stream"] == FLOAT_F32 else _round_to(total, 8, -125)
    y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / K + EPS) * (s["weight"].double() + c["offset"])
    out = [total, y if s["y"] is not None else None]
    if c["act"] == BF16:
        return out
    blocks = _round_to(y, 8, -125).view(M, K // 32, 32)
    code = _codes64(blocks, c["rule"])
    # the scaled values before they are rounded to 8 bits
    q = (blocks * torch.exp2(127 - code).unsqueeze(-1)).clamp(-448, 448).view(M, K)
    if c["act"] == T16:
        q, _ = _to_t16(q, code, M, K)
    return out + [q.reshape(-1), None]


def _exact_linear(s, c):
    N, K, dev = c["N"], c["K"], s["x"].device
    if c["act"] == BF16:
        a = s["x"].double()
    else:
        b = s["x"].double().view(-1, K // 32, 32)
        scale = _pow2(_codes64(b, c["rule"])).unsqueeze(-1)
        a = (_round_to(b / scale, 4, -5).clamp(-448, 448) * scale).view(-1, K)
    if c["elem"] == E4M3:
        w = _e4m3_table(dev)[s["w"].int()]
    else:
        w = torch.stack([_e2m1_table(dev)[(s["w"] % 16).int()], _e2m1_table(dev)[(s["w"] // 16).int()]], 2)
    k = _pow2(s["codes"])
    if c["layout"] == BLK32:
        k = k.repeat_interleave(32, dim=0)
    z = torch.mm(a, (w.reshape(N, K // 32, 32) * k.unsqueeze(-1)).view(N, K).t())
    if s["bias"] is not None:
        z += s["bias"].double()
    g = z[:, 0::2] if c["gated"] else z
    if c["fn"] in ("relu", "relu2"):
        h = torch.where(g > 0, g, 0.0)
        h = h * h if c["fn"] == "relu2" else h
    elif c["fn"] == "silu":
        h = g * torch.sigmoid(g)
    elif c["fn"] == "gelu":
        h = g * torch.special.ndtr(g)
    elif c["fn"] == "gelu_tanh":
        h = 0.5 * g * (1 + torch.tanh((2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    else:
        h = g
    if c["gated"]:
        h = h * z[:, 1::2]
    return h + s["residual"].double() if s["residual"] is not None else h


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, norm=_exact_norm, linear=_exact_linear)[case["op"]](s, case)
