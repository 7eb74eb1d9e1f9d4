// mx_ops_api.cpp -- the C ABI (include/mx.h) of the operators around the
// linear: residual norm, expert sort, grouped products, combine, adapters.
// Validation is pure host code and runs before any device call.
#include <hip/hip_runtime.h>

#include "mx_host.h"

namespace {

using namespace mx;

bool ld_bad(int64_t ld, int64_t cols) { return ld < cols || ld > kMaxLd; }

hipStream_t hip(mx_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

mx_status mx_add_rms_norm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *residual,
                          int64_t ldr, const void *weight, float eps, int act, int rule, void *sum,
                          int64_t lds, void *y, int64_t ldy, void *xq, int64_t ldq, void *xcodes,
                          int64_t ldc, mx_stream_t stream) {
    if (act != ACT_BF16 && act != ACT_MXFP8 && act != ACT_MXFP8_T16) return MX_ERR_UNSUPPORTED;
    if (rule != RULE_OCP && rule != RULE_CEIL448) return MX_ERR_UNSUPPORTED;
    if (M < 1 || M > kMaxRows || K < 32 || K % 32 != 0 || K > kNormMaxK || !(eps >= 0.0f))
        return MX_ERR_SHAPE;
    if (!x || !weight) return MX_ERR_NULL;
    if (ld_bad(ldx, K) || (residual && ld_bad(ldr, K)) || (sum && ld_bad(lds, K)) ||
        (y && ld_bad(ldy, K)))
        return MX_ERR_SHAPE;
    if (act == ACT_BF16 ? !y : (!xq || !xcodes)) return MX_ERR_NULL;
    if (act == ACT_MXFP8 && (ld_bad(ldq, K) || ld_bad(ldc, K / 32))) return MX_ERR_SHAPE;
    if (!aligned16(x) || ldx % 8 != 0 || !aligned16(weight) ||
        (residual && (!aligned16(residual) || ldr % 8 != 0)) ||
        (sum && (!aligned16(sum) || lds % 8 != 0)) || (y && (!aligned16(y) || ldy % 8 != 0)))
        return MX_ERR_ALIGN;
    if (act != ACT_BF16 && (!aligned16(xq) || (act == ACT_MXFP8 && ldq % 16 != 0) ||
                            (act == ACT_MXFP8_T16 && !aligned16(xcodes))))
        return MX_ERR_ALIGN;
    const Span sx{x, M, ldx, K, 2}, sr{residual, M, ldr, K, 2}, sw{weight, 1, K, K, 2};
    const Span ss{sum, M, lds, K, 2}, sy{y, M, ldy, K, 2};
    Span sq{nullptr, 1, 0, 0, 1}, sc{nullptr, 1, 0, 0, 1};
    if (act == ACT_MXFP8) {
        sq = {xq, M, ldq, K, 1};
        sc = {xcodes, M, ldc, K / 32, 1};
    } else if (act == ACT_MXFP8_T16) {
        sq = {xq, 1, 0, act_t16_data_bytes(M, K), 1};
        sc = {xcodes, 1, 0, act_codes_t16_bytes(M, K), 1};
    }
    if (!apart_or_same(ss, sx) || !apart_or_same(ss, sr) || !apart_or_same(sy, sx) ||
        !apart_or_same(sy, sr) || overlap(ss, sy))
        return MX_ERR_UNSUPPORTED;
    for (const Span &out : {ss, sy, sq, sc})
        if (overlap(out, sw)) return MX_ERR_UNSUPPORTED;
    for (const Span &out : {sq, sc})
        if (overlap(out, sx) || overlap(out, sr) || overlap(out, ss) || overlap(out, sy))
            return MX_ERR_UNSUPPORTED;
    if (overlap(sq, sc)) return MX_ERR_UNSUPPORTED;
    mx_status st = device_ok();
    if (st != MX_OK) return st;
    NormArgs a{};
    a.M = M;
    a.K = K;
    a.x = static_cast<const uint16_t *>(x);
    a.ldx = ldx;
    a.res = static_cast<const uint16_t *>(residual);
    a.ldr = ldr;
    a.weight = static_cast<const uint16_t *>(weight);
    a.eps = eps;
    a.sum = static_cast<uint16_t *>(sum);
    a.lds = lds;
    a.y = static_cast<uint16_t *>(y);
    a.ldy = ldy;
    a.xq = static_cast<uint8_t *>(xq);
    a.ldq = ldq;
    a.xcodes = static_cast<uint8_t *>(xcodes);
    a.ldc = ldc;
    log_dispatch("add_rms_norm: add_rms_norm_kernel, %s output (rule %d); M=%lld K=%lld",
                 act == ACT_BF16 ? "bf16" : act == ACT_MXFP8 ? "row-major MXFP8" : "T16", rule,
                 (long long)M, (long long)K);
    return launched(launch_add_rms_norm(a, act, rule, hip(stream)));
}

mx_status mx_moe_sort_workspace(int64_t E, int64_t T, int64_t topk, size_t *bytes) {
    if (!bytes) return MX_ERR_NULL;
    if (E < 1 || E > kSortMaxExperts || T < 1 || topk < 1 || topk > E || T > kMaxRows / topk)
        return MX_ERR_SHAPE;
    *bytes = (size_t)moe_sort_ws_bytes(E, T * topk);
    return MX_OK;
}

mx_status mx_moe_sort(int64_t E, int64_t T, int64_t topk, const int32_t *topk_ids,
                      int32_t *offsets, int32_t *rows, int32_t *pos, void *ws, size_t ws_bytes,
                      mx_stream_t stream) {
    size_t need = 0;
    mx_status st = mx_moe_sort_workspace(E, T, topk, &need);
    if (st != MX_OK) return st;
    if (!topk_ids || !offsets || !rows || !pos) return MX_ERR_NULL;
    if (!aligned4(topk_ids) || !aligned4(offsets) || !aligned4(rows) || !aligned4(pos))
        return MX_ERR_ALIGN;
    if (need > 0 && (!ws || ws_bytes < need)) return MX_ERR_WORKSPACE;
    if (need > 0 && !aligned16(ws)) return MX_ERR_ALIGN;
    const int64_t P = T * topk;
    const Span in{topk_ids, 1, 0, P, 4}, so{offsets, 1, 0, E + 1, 4}, sr{rows, 1, 0, P, 4},
        sp{pos, 1, 0, P, 4}, sw{need ? ws : nullptr, 1, 0, (int64_t)need, 1};
    if (overlap(in, so) || overlap(in, sr) || overlap(in, sp) || overlap(in, sw) ||
        overlap(so, sr) || overlap(so, sp) || overlap(so, sw) || overlap(sr, sp) ||
        overlap(sr, sw) || overlap(sp, sw))
        return MX_ERR_UNSUPPORTED;
    if ((st = device_ok()) != MX_OK) return st;
    log_dispatch("moe_sort: %smoe_place_kernel; E=%lld T=%lld topk=%lld",
                 need ? "moe_count_kernel, " : "", (long long)E, (long long)T, (long long)topk);
    return launched(launch_moe_sort(E, P, topk, topk_ids, offsets, rows, pos, ws, hip(stream)));
}

mx_status mx_grouped_workspace(int elem, int layout, int64_t E, int64_t N, int64_t K, int64_t M,
                               int act, int prequantized, size_t *bytes) {
    if (!bytes) return MX_ERR_NULL;
    mx_status st = shape_ok(elem, layout, E, N, K);
    if (st != MX_OK) return st;
    if (act != ACT_MXFP8 && act != ACT_MXFP8_T16) return MX_ERR_UNSUPPORTED;
    if (elem == E2M1 && layout != ROW32) return MX_ERR_UNSUPPORTED;
    if (E > kMaxExperts || M < 1 || M > kMaxRows) return MX_ERR_SHAPE;
    // 32-bit offsets into one expert's weights and into a batch's tokens
    const int64_t kp = (K + 127) / 128 * 128;
    if (kp > kMaxRsrc / 272 || N > kMaxRsrc / kp || act_t16_data_bytes(M, K) > kMaxT16Bytes)
        return MX_ERR_SHAPE;
    (void)prequantized;                                   // staged into T16 either way
    *bytes = act == ACT_MXFP8
                 ? (size_t)(round256(act_t16_data_bytes(M, K)) + act_codes_t16_bytes(M, K))
                 : 0;
    return MX_OK;
}

mx_status mx_grouped_linear(int elem, int layout, int64_t E, int64_t N, int64_t K,
                            const void *w_packed, const void *codes_packed, int64_t M,
                            const int32_t *offsets, int act, int rule, int64_t xrows,
                            const void *x, int64_t ldx, const void *xq, int64_t ldq,
                            const void *xcodes, int64_t ldc, const int32_t *rows, int epi, void *y,
                            int64_t ldy, void *ws, size_t ws_bytes, mx_stream_t stream) {
    const bool given = xq && xcodes;
    size_t need = 0;
    mx_status st = mx_grouped_workspace(elem, layout, E, N, K, M, act, given ? 1 : 0, &need);
    if (st != MX_OK) return st;
    if (rule != RULE_OCP && rule != RULE_CEIL448) return MX_ERR_UNSUPPORTED;
    if (epi != MX_EPI_NONE && epi != MX_EPI_SILU) return MX_ERR_UNSUPPORTED;
    const int64_t width = epi == MX_EPI_SILU ? N / 2 : N;
    if (ldy < width || ldy > kMaxRsrc / 512) return MX_ERR_SHAPE;   // 32-bit offsets: 256 rows of y
    if (!w_packed || !codes_packed || !offsets || !y) return MX_ERR_NULL;
    if (!aligned16(w_packed) || !aligned16(codes_packed) || !aligned4(offsets) ||
        !aligned16(y) || ldy % 8 != 0)
        return MX_ERR_ALIGN;
    if (act == ACT_MXFP8_T16) {
        if (!given) return MX_ERR_NULL;
        if (rows) return MX_ERR_UNSUPPORTED;              // T16 rows are in place already
        if (!aligned16(xq) || !aligned16(xcodes)) return MX_ERR_ALIGN;
    } else {
        if (xrows < 1 || xrows > kMaxRows || (!rows && xrows < M)) return MX_ERR_SHAPE;
        if (rows && !aligned4(rows)) return MX_ERR_ALIGN;
        if (given) {
            if (ld_bad(ldq, K) || ld_bad(ldc, K / 32)) return MX_ERR_SHAPE;
            if (!aligned16(xq) || ldq % 16 != 0) return MX_ERR_ALIGN;
        } else {
            if (!x) return MX_ERR_NULL;
            if (ld_bad(ldx, K)) return MX_ERR_SHAPE;
            if (!aligned16(x) || ldx % 8 != 0) return MX_ERR_ALIGN;
        }
        if (!ws || ws_bytes < need) return MX_ERR_WORKSPACE;
        if (!aligned16(ws)) return MX_ERR_ALIGN;
    }
    const Span sy{y, M, ldy, width, 2};
    size_t wb = 0, cb = 0;
    if ((st = mx_packed_sizes(elem, layout, E, N, K, &wb, &cb)) != MX_OK) return st;
    const Span ins[] = {
        {w_packed, 1, 0, (int64_t)wb, 1},
        {codes_packed, 1, 0, (int64_t)cb, 1},
        {act == ACT_MXFP8 && !given ? x : nullptr, xrows, ldx, K, 2},
        {act == ACT_MXFP8 && given ? xq : nullptr, xrows, ldq, K, 1},
        {act == ACT_MXFP8 && given ? xcodes : nullptr, xrows, ldc, K / 32, 1},
        {act == ACT_MXFP8_T16 ? xq : nullptr, 1, 0, act_t16_data_bytes(M, K), 1},
        {act == ACT_MXFP8_T16 ? xcodes : nullptr, 1, 0, act_codes_t16_bytes(M, K), 1},
        {rows, 1, 0, M, 4},
        {offsets, 1, 0, E + 1, 4}};
    const Span sw{need ? ws : nullptr, 1, 0, (int64_t)need, 1};
    for (const Span &in : ins)
        if (overlap(sy, in) || overlap(sw, in)) return MX_ERR_UNSUPPORTED;
    if (overlap(sy, sw)) return MX_ERR_UNSUPPORTED;
    if ((st = device_ok()) != MX_OK) return st;
    GroupedArgs g{};
    g.w = static_cast<const uint8_t *>(w_packed);
    g.codes = static_cast<const uint8_t *>(codes_packed);
    g.E = E;
    g.N = N;
    g.K = K;
    g.M = M;
    g.offsets = offsets;
    g.xq = static_cast<const uint8_t *>(xq);
    g.xct = static_cast<const uint8_t *>(xcodes);
    g.y = static_cast<uint16_t *>(y);
    g.ldy = ldy;
    g.epi = epi;
    g.invariant = batch_invariant() ? 1 : 0;
    if (act == ACT_MXFP8) {
        uint8_t *data = static_cast<uint8_t *>(ws);
        uint8_t *codes = data + round256(act_t16_data_bytes(M, K));
        StageArgs s{};
        s.M = M;
        s.K = K;
        s.E = E;
        s.xrows = xrows;
        s.offsets = offsets;
        s.rows = rows;
        if (given) {
            s.xq = g.xq;
            s.ldq = ldq;
            s.xc = g.xct;
            s.ldc = ldc;
        } else {
            s.x = static_cast<const uint16_t *>(x);
            s.ldx = ldx;
        }
        s.out = data;
        s.outc = codes;
        log_dispatch("grouped: stage_rows_kernel, %s rows%s; M=%lld K=%lld",
                     given ? "row-major MXFP8" : "bf16", rows ? " by index" : "", (long long)M,
                     (long long)K);
        if ((st = launched(launch_stage_rows(s, rule, hip(stream)))) != MX_OK) return st;
        g.xq = data;
        g.xct = codes;
    }
    log_dispatch("grouped: %s %s%s; E=%lld M=%lld N=%lld K=%lld", grouped_kernel_name(g),
                 elem == E4M3 ? "E4M3" : "E2M1", epi ? " silu" : "", (long long)E, (long long)M,
                 (long long)N, (long long)K);
    return launched(launch_grouped(elem, layout, g, hip(stream)));
}

mx_status mx_moe_combine(int64_t T, int64_t topk, int64_t N, int64_t M, const void *ys,
                         int64_t ldys, const int32_t *pos, const float *topk_weights, void *y,
                         int64_t ldy, mx_stream_t stream) {
    if (T < 1 || topk < 1 || T > kMaxRows / topk || M < 1 || M > kMaxRows || N < 8 ||
        N % 8 != 0 || N > kCombineMaxCols ||
        ld_bad(ldys, N) || ld_bad(ldy, N))
        return MX_ERR_SHAPE;
    if (!ys || !pos || !topk_weights || !y) return MX_ERR_NULL;
    if (!aligned16(ys) || ldys % 8 != 0 || !aligned4(pos) || !aligned4(topk_weights) ||
        !aligned16(y) || ldy % 8 != 0)
        return MX_ERR_ALIGN;
    const Span sy{y, T, ldy, N, 2};
    const Span ins[] = {{ys, M, ldys, N, 2}, {pos, 1, 0, T * topk, 4},
                        {topk_weights, 1, 0, T * topk, 4}};
    for (const Span &in : ins)
        if (overlap(sy, in)) return MX_ERR_UNSUPPORTED;
    mx_status st = device_ok();
    if (st != MX_OK) return st;
    log_dispatch("moe_combine: moe_gather_sum_kernel; T=%lld topk=%lld N=%lld", (long long)T,
                 (long long)topk, (long long)N);
    return launched(launch_moe_gather_sum(T, topk, N, M, static_cast<const uint16_t *>(ys), ldys,
                                          pos, topk_weights, static_cast<uint16_t *>(y), ldy,
                                          hip(stream)));
}

// the adapters' workspace in a given batch-invariant mode
static mx_status lora_bytes(int64_t L, int64_t R, int64_t N, int64_t K, int64_t M, bool invariant,
                            size_t *bytes) {
    if (L < 1 || L > kMaxRows || R < 8 || R % 8 != 0 || R > kLoraMaxRank || N < 16 ||
        N % 16 != 0 || K < 32 || K % 32 != 0 || M < 1 || M > kMaxRows ||
        N > kLoraMaxCols || K > kLoraMaxK)
        return MX_ERR_SHAPE;
    // 32-bit offsets into one adapter's matrices
    if (K > kMaxRsrc / (2 * R) || N > kMaxRsrc / (2 * R)) return MX_ERR_SHAPE;
    *bytes = (size_t)(lora_splits(M, K, invariant) * M * ((R + 15) / 16 * 16) * 4);
    return MX_OK;
}

mx_status mx_lora_workspace(int64_t L, int64_t R, int64_t N, int64_t K, int64_t M, size_t *bytes) {
    if (!bytes) return MX_ERR_NULL;
    return lora_bytes(L, R, N, K, M, batch_invariant(), bytes);
}

mx_status mx_lora_add(int64_t L, int64_t R, int64_t N, int64_t K, const void *a, const void *b,
                      const float *scales, int64_t M, const void *x, int64_t ldx,
                      const int32_t *ids, const void *base, int64_t ldb, void *y, int64_t ldy,
                      void *ws, size_t ws_bytes, mx_stream_t stream) {
    size_t need = 0;
    // read once: the launch writes what the size checked here has room for, also
    // when another thread changes the mode meanwhile
    const bool invariant = batch_invariant();
    mx_status st = lora_bytes(L, R, N, K, M, invariant, &need);
    if (st != MX_OK) return st;
    if (ldx < K || ldb < N || ldy < N) return MX_ERR_SHAPE;
    // 32-bit offsets into a tile of 64 rows
    if (ldx > kMaxRsrc / 128 || ldb > kMaxRsrc / 128 || ldy > kMaxRsrc / 128) return MX_ERR_SHAPE;
    if (!a || !b || !x || !ids || !base || !y) return MX_ERR_NULL;
    if (!aligned16(a) || !aligned16(b) || !aligned16(x) || ldx % 8 != 0 || !aligned16(base) ||
        ldb % 8 != 0 || !aligned16(y) || ldy % 8 != 0 || !aligned4(ids) ||
        (scales && !aligned4(scales)))
        return MX_ERR_ALIGN;
    if (!ws || ws_bytes < need) return MX_ERR_WORKSPACE;
    if (!aligned16(ws)) return MX_ERR_ALIGN;
    const Span sy{y, M, ldy, N, 2}, sb{base, M, ldb, N, 2}, sw{ws, 1, 0, (int64_t)need, 1};
    const Span ins[] = {{a, 1, 0, L * R * K, 2}, {b, 1, 0, L * N * R, 2}, {x, M, ldx, K, 2},
                        {ids, 1, 0, M, 4}, {scales, 1, 0, L, 4}};
    for (const Span &in : ins)
        if (overlap(sy, in) || overlap(sw, in)) return MX_ERR_UNSUPPORTED;
    if (!apart_or_same(sy, sb) || overlap(sw, sb) || overlap(sw, sy)) return MX_ERR_UNSUPPORTED;
    if ((st = device_ok()) != MX_OK) return st;
    LoraArgs g{};
    g.L = L;
    g.R = R;
    g.N = N;
    g.K = K;
    g.M = M;
    g.a = static_cast<const uint16_t *>(a);
    g.b = static_cast<const uint16_t *>(b);
    g.scales = scales;
    g.x = static_cast<const uint16_t *>(x);
    g.ldx = ldx;
    g.ids = ids;
    g.base = static_cast<const uint16_t *>(base);
    g.ldb = ldb;
    g.y = static_cast<uint16_t *>(y);
    g.ldy = ldy;
    g.ws = static_cast<float *>(ws);
    g.invariant = invariant;
    log_dispatch("lora: lora_shrink_kernel, lora_expand_kernel; L=%lld R=%lld M=%lld N=%lld K=%lld",
                 (long long)L, (long long)R, (long long)M, (long long)N, (long long)K);
    return launched(launch_lora(g, hip(stream)));
}

}  // extern "C"
