"""Measured cases of the operators around the block-scaled linear layer.

Five operators that a serving program runs next to ``mx_linear``:

* ``add_rms_norm``    residual addition, root-mean-square norm and MXFP8 output
* ``moe_sort``        routed (token, choice) pairs put in expert order
* ``grouped_linear``  matrix products grouped by expert with ragged row counts
* ``moe_combine``     weighted sum of a token's expert outputs
* ``lora_add``        low-rank adapters of many requests beside a projection

A case is a dict of plain values.  ``prepare`` makes what the program holds
before the call (activations, packed weights, routing, output buffers) on the
GPU, from the seed alone; ``run`` is one call.  With ``own`` false, ``run``
computes the operator in elementary torch operations in 32 bits; with ``own``
true it calls the library.  ``exact`` computes it in 64 bits.

What is held in 8 bits comes back as torch's 8-bit floating types: e4m3 values
and E8M0 scales, in the layout that the call fills.
"""
from __future__ import annotations

import torch

own = False

E4M3, E2M1 = 0, 1
ROW32, BLK32 = 0, 1
OCP, CEIL448 = 0, 1
MXFP8, T16 = 1, 2
EPS = 1e-6


def listed():
    return [
        # decode: the norm ahead of a quantized projection, a few tokens, fed to
        # the matrix cores' tile layout (latency)
        dict(name="norm_decode_t16", op="norm", M=4, K=7168, act=T16, rule=OCP, keep=False),
        # prefill: row-major bytes for the experts' gather, and the bf16 rows
        # that the router reads
        dict(name="norm_prefill_rows", op="norm", M=4096, K=7168, act=MXFP8, rule=OCP, keep=True),
        # decode: gate and up products of 16 tokens over 32 experts of e2m1
        # weights (the weights' stream)
        dict(name="grouped_w4_decode_gate_up", op="grouped", elem=E2M1, layout=ROW32, E=32,
             N=4096, K=4096, T=16, topk=8, form="bf16", gather=True, silu=True, rule=OCP,
             skew=0.5, drop=0.0),
        # a short prompt in odd sizes: uneven experts, padding tokens that no
        # expert takes, rows quantized ahead of the call
        dict(name="grouped_w8_ragged", op="grouped", elem=E4M3, layout=BLK32, E=24, N=4096,
             K=1568, T=517, topk=4, form="mxfp8", gather=True, silu=False, rule=CEIL448,
             skew=1.5, drop=0.1),
        # prefill: gate and up products of a long prompt, e2m1 weights
        dict(name="grouped_w4_prefill_gate_up", op="grouped", elem=E2M1, layout=ROW32, E=32,
             N=4096, K=4096, T=2048, topk=8, form="bf16", gather=True, silu=True, rule=OCP,
             skew=0.5, drop=0.0),
        # prefill: down projection of the hidden rows, e4m3 weights
        dict(name="grouped_w8_prefill_down", op="grouped", elem=E4M3, layout=ROW32, E=32,
             N=7168, K=2048, T=4096, topk=8, form="bf16", gather=False, silu=False, rule=OCP,
             skew=0.5, drop=0.0),
        # the routing's order for a decode step and for a large prefill batch
        dict(name="sort_decode", op="sort", E=32, T=16, topk=8, drop=0.0, skew=0.5),
        dict(name="sort_prefill", op="sort", E=128, T=16384, topk=8, drop=0.05, skew=1.0),
        # the experts' outputs summed per token, decode and prefill
        dict(name="combine_decode", op="combine", E=32, T=16, topk=8, N=7168, drop=0.0),
        dict(name="combine_prefill", op="combine", E=32, T=4096, topk=8, N=7168, drop=0.05),
        # decode: 16 requests, most with an adapter of their own
        dict(name="lora_decode", op="lora", L=32, R=16, N=7168, K=7168, M=16, run=1, none=0.1),
        # prefill: a batch of prompts, each with its request's adapter
        dict(name="lora_prefill", op="lora", L=8, R=64, N=4096, K=7168, M=4096, run=700,
             none=0.1),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "grouped", "grouped", "sort", "combine", "lora"])
    if op == "norm":
        return dict(op=op, M=_between(rng, 1, 4096), K=32 * _between(rng, 1, 256),
                    act=rng.choice([MXFP8, T16]), rule=rng.choice([OCP, CEIL448]),
                    keep=rng.random() < 0.5)
    if op == "grouped":
        elem = rng.choice([E4M3, E2M1])
        E = _between(rng, 1, 64)
        topk = min(E, rng.randint(1, 8))
        T = _between(rng, 1, max(1, 16384 // topk))
        return dict(op=op, elem=elem, layout=rng.choice([ROW32, BLK32]) if elem == E4M3 else ROW32,
                    E=E, N=32 * _between(rng, 1, 128), K=32 * _between(rng, 1, 128), T=T,
                    topk=topk, form=rng.choice(["bf16", "mxfp8"]), gather=rng.random() < 0.7,
                    silu=rng.random() < 0.5, rule=rng.choice([OCP, CEIL448]),
                    skew=rng.choice([0.0, 0.5, 1.5]), drop=rng.choice([0.0, 0.2]))
    if op == "sort":
        E = _between(rng, 1, 256)
        return dict(op=op, E=E, T=_between(rng, 1, 16384), topk=min(E, rng.randint(1, 8)),
                    drop=rng.choice([0.0, 0.1]), skew=rng.choice([0.0, 1.0, 2.0]))
    if op == "combine":
        return dict(op=op, E=32, T=_between(rng, 1, 4096), topk=rng.randint(1, 8),
                    N=8 * _between(rng, 8, 896), drop=rng.choice([0.0, 0.2]))
    M = _between(rng, 1, 4096)
    return dict(op=op, L=_between(rng, 1, 64), R=rng.choice([8, 16, 24, 32, 64]),
                N=16 * _between(rng, 4, 448), K=32 * _between(rng, 2, 224), M=M,
                run=_between(rng, 1, max(1, M // 2)), none=rng.choice([0.0, 0.2]))


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

    def routing(self, E, T, topk, skew, drop):
        """Top-k ids [T, topk] (int32) of normal logits, `skew` times a normal
        preference per expert added; a share `drop` of the tokens (padding of a
        batch) takes no expert: id -1.  Softmax weights of the chosen logits."""
        logits = self.normal(T, E) + skew * self.normal(E)
        val, ids = logits.topk(topk, dim=1)
        gone = self.uniform(T, 1) < drop
        return ids.masked_fill(gone, -1).to(torch.int32), torch.softmax(val, dim=1)

    def weight(self, elem, layout, E, N, K):
        """A normal weight in the elements' format: standard bytes
        [E, N, K or K/2] and codes [E*N, K/32] or [E*N/32, K/32]."""
        w = self.normal(E, N, K // 32, 32).mul_(0.02)
        amax = w.abs().amax(-1)                                     # [E, N, K/32]
        if layout == BLK32:
            amax = amax.view(E, N // 32, 32, K // 32).amax(2)
        bits = amax.contiguous().view(torch.int32)
        code = ((bits >> 23) - (8 if elem == E4M3 else 2)).clamp_(0, 254)
        row = code if layout == ROW32 else code.repeat_interleave(32, dim=1)
        w.mul_(((254 - row) << 23).to(torch.int32).view(torch.float32).unsqueeze(-1))
        code = code.to(torch.uint8).view(-1, K // 32)
        if elem == E4M3:
            return w.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(E, N, K), code
        edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=self.device)
        nib = torch.bucketize(w.abs(), edge, out_int32=True).to(torch.uint8)
        nib += (w < 0).to(torch.uint8) * 8
        nib = nib.view(E, N, K // 2, 2)
        return nib[..., 0] | nib[..., 1] << 4, code


def _pack(elem, layout, E, N, K, w, codes):
    """The packed weight and codes that the library documents (what its load-time
    pack writes): 16-row tiles of 16-byte pieces; code dwords of four steps, a
    trailer with the smallest and largest code."""
    rowb = K if elem == E4M3 else K // 2
    wp = w.view(E, N // 16, 16, rowb // 16, 16).transpose(2, 3).contiguous().view(-1)
    Q = -(-K // 512)
    c = torch.full((codes.shape[0], 16 * Q), 128, dtype=torch.uint8, device=w.device)
    c[:, :K // 32] = codes
    if layout == ROW32:
        c = c.view(E * N // 16, 16, Q, 4, 4).permute(0, 2, 4, 1, 3)
    else:
        c = c.view(-1, Q, 4, 4).permute(0, 1, 3, 2)
    tail = torch.zeros(16, dtype=torch.uint8, device=w.device)
    tail[0], tail[1] = codes.min(), codes.max()
    return wp, torch.cat([c.reshape(-1), tail])


def _norm_state(c, i):
    M, K = c["M"], c["K"]
    channel = torch.where(i.uniform(K) < 0.01, 20.0, 1.0)     # a residual stream's large channels
    s = dict(x=i.normal(M, K).bfloat16(), residual=(2 * i.normal(M, K) * channel).bfloat16(),
             weight=(1 + 0.2 * i.normal(K)).bfloat16())
    s["sum"] = torch.empty_like(s["x"])
    s["y"] = torch.empty_like(s["x"]) if c["keep"] else None
    S = -(-K // 128)
    n, m = ((M * K, M * (K // 32)) if c["act"] == MXFP8 else
            (-(-M // 16) * S * 2048, -(-M // 16) * (-(-S // 4)) * 256))
    s["xq"] = torch.empty(n, dtype=torch.uint8, device=i.device)
    s["xcodes"] = torch.empty(m, dtype=torch.uint8, device=i.device)
    return s


def _order(ids, E):
    """Pairs in expert order: (offsets [E + 1], token of each place, place of
    each pair), -1 behind the last pair and for pairs without an expert."""
    T, topk = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, order = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    place = torch.arange(T * topk, device=ids.device)
    rows = torch.where(key < E, order // topk, -1).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = torch.where(key < E, place, -1)
    return offsets, rows, pos.to(torch.int32).view(T, topk)


def _grouped_state(c, i):
    E, N, K, T, topk = c["E"], c["N"], c["K"], c["T"], c["topk"]
    w, codes = i.weight(c["elem"], c["layout"], E, N, K)
    ids, _ = i.routing(E, T, topk, c["skew"], c["drop"])
    offsets, rows, _ = _order(ids, E)
    M = T * topk
    xrows = T if c["gather"] else M
    s = dict(w=w, codes=codes, M=M, xrows=xrows, offsets=offsets,
             rows=rows if c["gather"] else None,
             most=int((offsets[1:] - offsets[:-1]).max()))
    s["w_packed"], s["codes_packed"] = _pack(c["elem"], c["layout"], E, N, K, w, codes)
    x = i.normal(xrows, K)
    x = torch.where(i.uniform(xrows, K) < 0.01, 20 * x, x).bfloat16()
    if c["form"] == "bf16":
        s["x"] = x
    else:
        q, code = _quantize(x.float(), c["rule"])
        pad = torch.zeros(xrows, (K + 15) // 16 * 16, dtype=torch.uint8, device=i.device)
        pad[:, :K] = q.view(torch.uint8)
        s["xq"], s["xcodes"] = pad, code.contiguous()
    # rows that no expert takes keep what the buffer held: zeros here
    s["y"] = torch.zeros(M, N // 2 if c["silu"] else N, dtype=torch.bfloat16, device=i.device)
    return s


def _sort_state(c, i):
    ids, _ = i.routing(c["E"], c["T"], c["topk"], c["skew"], c["drop"])
    new = lambda n: torch.empty(n, dtype=torch.int32, device=i.device)  # noqa: E731
    return dict(ids=ids, offsets=new(c["E"] + 1), rows=new(ids.numel()), pos=new(ids.shape))


def _combine_state(c, i):
    ids, weights = i.routing(c["E"], c["T"], c["topk"], 0.5, c["drop"])
    _, _, pos = _order(ids, c["E"])
    return dict(pos=pos, weights=weights.float().contiguous(),
                ys=i.normal(c["T"] * c["topk"], c["N"]).bfloat16(),
                y=torch.empty(c["T"], c["N"], dtype=torch.bfloat16, device=i.device))


def _lora_state(c, i):
    L, R, N, K, M = c["L"], c["R"], c["N"], c["K"], c["M"]
    # a request's rows are neighbours and share its adapter
    starts = (i.uniform(M) < 1.0 / c["run"]).long().cumsum(0)
    adapter = (i.uniform(M + 1) * L).long().clamp_(0, L - 1)
    adapter = torch.where(i.uniform(M + 1) < c["none"], -1, adapter)
    return dict(a=(i.normal(L, R, K) / K ** 0.5).bfloat16(),
                b=(i.normal(L, N, R) / R ** 0.5).bfloat16(),
                scales=0.5 + i.uniform(L), ids=adapter[starts].to(torch.int32),
                x=i.normal(M, K).bfloat16(), base=i.normal(M, N).bfloat16(),
                y=torch.empty(M, N, dtype=torch.bfloat16, device=i.device))


def prepare(case, seed):
    make = dict(norm=_norm_state, grouped=_grouped_state, sort=_sort_state,
                combine=_combine_state, lora=_lora_state)[case["op"]]
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


def _norm(s, c):
    f = (s["x"].float() + s["residual"].float()).bfloat16()
    v = f.float()
    y = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()).bfloat16()
    q, code = _quantize(y.float(), c["rule"])
    q, code = q.view(torch.uint8), code
    if c["act"] == T16:
        q, code = _to_t16(q, code, c["M"], c["K"])
    return [f, y if c["keep"] else None, q.reshape(-1).view(torch.float8_e4m3fn),
            code.reshape(-1).view(torch.float8_e8m0fnu)]


def _weights32(s, c):
    E, N, K = c["E"], c["N"], c["K"]
    if c["elem"] == E4M3:
        w = s["w"].view(torch.float8_e4m3fn).float()
    else:
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                             device=s["w"].device)
        w = torch.stack([value[(s["w"] & 15).int()], value[(s["w"] >> 4).int()]], -1)
    scale = (s["codes"].int() << 23).view(torch.float32).view(E, -1, K // 32)
    if c["layout"] == BLK32:
        scale = scale.repeat_interleave(32, dim=1)
    return (w.view(E, N, K // 32, 32) * scale.unsqueeze(-1)).view(E, N, K)


def _grouped(s, c):
    E, K, M = c["E"], c["K"], s["M"]
    if c["form"] == "bf16":
        q, code = _quantize(s["x"].float(), c["rule"])
    else:
        q, code = s["xq"][:, :K].view(torch.float8_e4m3fn), s["xcodes"]
    a = (q.float().view(-1, K // 32, 32) *
         (code.int() << 23).view(torch.float32).unsqueeze(-1)).view(-1, K)
    # one padded batch of products: place p of expert e is row offsets[e] + p
    first = s["offsets"][:E].long().unsqueeze(1)
    count = s["offsets"][1:].long().unsqueeze(1) - first
    p = torch.arange(s["most"], device=a.device)
    place = torch.where(p < count, first + p, M)                 # [E, most]
    row = torch.arange(M, device=a.device) if s["rows"] is None else s["rows"].long()
    row = torch.cat([row, row.new_zeros(1)])
    prod = torch.bmm(a[row[place].clamp_min(0)], _weights32(s, c).transpose(1, 2))
    if c["silu"]:
        g, u = prod[..., 0::2], prod[..., 1::2]
        prod = g / (1 + torch.exp(-g)) * u
    y = torch.zeros(M + 1, prod.shape[-1], dtype=torch.bfloat16, device=a.device)
    y[place.reshape(-1)] = prod.bfloat16().view(-1, prod.shape[-1])
    y[M] = 0
    return y[:M]


def _combine(s, c):
    pos = s["pos"].long()
    w = torch.where(pos >= 0, s["weights"], 0.0)
    return (s["ys"][pos.clamp_min(0)].float() * w.unsqueeze(-1)).sum(1).bfloat16()


def _lora(s, c):
    L, R, N, M = c["L"], c["R"], c["N"], c["M"]
    mine = (s["ids"].unsqueeze(1) == torch.arange(L, device=s["x"].device)).float() * s["scales"]
    v = (s["x"].float() @ s["a"].float().view(L * R, -1).t()).view(M, L, R) * mine.unsqueeze(-1)
    d = v.view(M, L * R) @ s["b"].float().transpose(1, 2).reshape(L * R, N)
    return (s["base"].float() + d).bfloat16()


# ---- the library's calls --------------------------------------------------------------


def _own(s, c):
    import microscaling_quantized_linear_amd as mx

    op = c["op"]
    if op == "norm":
        M, K, y = c["M"], c["K"], s["y"]
        mx.mx_add_rms_norm(M, K, s["x"], K, s["residual"], K, s["weight"], EPS, c["act"],
                           c["rule"], s["sum"], K, y, K if y is not None else 0, s["xq"], K,
                           s["xcodes"], K // 32)
        return [s["sum"], y, s["xq"].view(torch.float8_e4m3fn),
                s["xcodes"].view(torch.float8_e8m0fnu)]
    if op == "grouped":
        E, N, K, M, y = c["E"], c["N"], c["K"], s["M"], s["y"]
        given = c["form"] == "mxfp8"
        ws = s.get("ws")
        if ws is None:                     # kept by the program for its next calls
            need = mx.mx_grouped_workspace(c["elem"], c["layout"], E, N, K, M, MXFP8, given)
            ws = s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=y.device)
        mx.mx_grouped_linear(c["elem"], c["layout"], E, N, K, s["w_packed"], s["codes_packed"], M,
                             s["offsets"], MXFP8, c["rule"], s["xrows"], s.get("x"),
                             0 if given else K, s.get("xq"), s["xq"].shape[1] if given else 0,
                             s.get("xcodes"), K // 32 if given else 0, s["rows"],
                             1 if c["silu"] else 0, y, y.shape[1], ws, ws.numel())
        return y
    if op == "sort":
        E, T, topk = c["E"], c["T"], c["topk"]
        ws = s.get("ws")
        if ws is None:
            need = mx.mx_moe_sort_workspace(E, T, topk)
            ws = s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["ids"].device)
        mx.mx_moe_sort(E, T, topk, s["ids"], s["offsets"], s["rows"], s["pos"], ws, ws.numel())
        return [s["offsets"], s["rows"], s["pos"]]
    if op == "combine":
        T, topk, N = c["T"], c["topk"], c["N"]
        mx.mx_moe_combine(T, topk, N, T * topk, s["ys"], N, s["pos"], s["weights"], s["y"], N)
        return s["y"]
    L, R, N, K, M = c["L"], c["R"], c["N"], c["K"], c["M"]
    ws = s.get("ws")
    if ws is None:
        need = mx.mx_lora_workspace(L, R, N, K, M)
        ws = s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["x"].device)
    mx.mx_lora_add(L, R, N, K, s["a"], s["b"], s["scales"], M, s["x"], K, s["ids"], s["base"], N,
                   s["y"], N, ws, ws.numel())
    return s["y"]


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "sort":
        return list(_order(state["ids"], c["E"]))
    return dict(norm=_norm, grouped=_grouped, combine=_combine, lora=_lora)[c["op"]](state, c)


def work(case):
    """Each input read once, each output written once; the products' operations."""
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        rows = -(-c["M"] // 16) * 16 if c["act"] == T16 else c["M"]
        return dict(bytes=n * (8 if c["keep"] else 6) + rows * c["K"] * 33 / 32 + 2 * c["K"],
                    flops=8 * n)
    if c["op"] == "grouped":
        E, N, K = c["E"], c["N"], c["K"]
        M = c["T"] * c["topk"] * (1 - c["drop"])
        used = E * (1 - (1 - 1 / E) ** M) if E > 1 else 1.0      # experts that get a row
        per = N * K * (1 if c["elem"] == E4M3 else 0.5)
        codes = N * K / 32 / (32 if c["layout"] == BLK32 else 1)
        x = (c["T"] if c["gather"] else c["T"] * c["topk"]) * K
        return dict(bytes=used * (per + codes) + x * (2 if c["form"] == "bf16" else 33 / 32) +
                    M * N * (1 if c["silu"] else 2), flops=2 * M * N * K)
    if c["op"] == "sort":
        return dict(bytes=12 * c["T"] * c["topk"] + 4 * c["E"], flops=0)
    if c["op"] == "combine":
        pairs = c["T"] * c["topk"] * (1 - c["drop"])
        return dict(bytes=2 * pairs * c["N"] + 2 * c["T"] * c["N"] + 8 * c["T"] * c["topk"],
                    flops=2 * pairs * c["N"])
    L, R, N, K, M = c["L"], c["R"], c["N"], c["K"], c["M"]
    live = M * (1 - c["none"])
    runs = max(1.0, M / c["run"]) * (1 - c["none"])
    used = L * (1 - (1 - 1 / L) ** runs) if L > 1 else 1.0
    return dict(bytes=used * 2 * R * (N + K) + 2 * live * K + 4 * M * N, flops=2 * live * R * (N + K))


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


def _round_bf16(v):
    """64-bit values rounded once, to nearest even, to 8 significant bits."""
    _, e = torch.frexp(v)
    step = torch.exp2(e.double().clamp_min(-125) - 8)
    return torch.round(v / step) * step


def _round_e4m3(v):
    _, e = torch.frexp(v)
    step = torch.exp2(e.double().clamp_min(-5) - 4)
    return (torch.round(v / step) * step).clamp(-448, 448)


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


def exact(case, seed):
    s, c = prepare(case, seed), case
    dev = _device()
    if c["op"] == "sort":
        return None
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        total = s["x"].double() + s["residual"].double()
        v = _round_bf16(total)
        y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / K + EPS) * s["weight"].double()
        blocks = _round_bf16(y).view(M, K // 32, 32)
        code = _codes64(blocks, c["rule"])
        # the scaled values before they are rounded to 8 bits
        q = (blocks * torch.exp2(127 - code).unsqueeze(-1)).clamp(-448, 448).view(M, K)
        if c["act"] == T16:
            q, _ = _to_t16(q, code, M, K)
        return [total, y if c["keep"] else None, q.reshape(-1), None]
    if c["op"] == "grouped":
        E, N, K, M = c["E"], c["N"], c["K"], s["M"]
        if c["form"] == "bf16":
            b = s["x"].double().view(-1, K // 32, 32)
            scale = _pow2(_codes64(b, c["rule"])).unsqueeze(-1)
            a = (_round_e4m3(b / scale) * scale).view(-1, K)
        else:
            a = _e4m3_table(dev)[s["xq"][:, :K].int()].view(-1, K // 32, 32)
            a = (a * _pow2(s["xcodes"]).unsqueeze(-1)).view(-1, K)
        out = torch.zeros(M, s["y"].shape[1], dtype=torch.float64, device=dev)
        codes = s["codes"].view(E, -1, K // 32)
        at = s["offsets"].tolist()
        for e in range(E):
            if at[e] == at[e + 1]:
                continue
            if c["elem"] == E4M3:
                w = _e4m3_table(dev)[s["w"][e].int()]
            else:
                w = torch.stack([_e2m1_table(dev)[(s["w"][e] % 16).int()],
                                 _e2m1_table(dev)[(s["w"][e] // 16).int()]], 2)
            k = _pow2(codes[e])
            if c["layout"] == BLK32:
                k = k.repeat_interleave(32, dim=0)
            w = (w.reshape(N, K // 32, 32) * k.unsqueeze(-1)).view(N, K)
            rows = slice(at[e], at[e + 1])
            r = a[rows] if s["rows"] is None else a[s["rows"][rows].long()]
            p = torch.mm(r, w.t())
            if c["silu"]:
                p = p[:, 0::2] * torch.sigmoid(p[:, 0::2]) * p[:, 1::2]
            out[rows] = p
        return out
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=dev)
        for k in range(c["topk"]):
            pos = s["pos"][:, k].long()
            live = (pos >= 0).double() * s["weights"][:, k].double()
            out += s["ys"][pos.clamp_min(0)].double() * live.unsqueeze(1)
        return out
    out = s["base"].double()
    for k in range(c["L"]):
        rows = torch.nonzero(s["ids"] == k).view(-1)
        if rows.numel():
            v = torch.mm(s["x"][rows].double(), s["a"][k].double().t())
            out[rows] += torch.mm(v, s["b"][k].double().t()) * s["scales"][k].double()
    return out
