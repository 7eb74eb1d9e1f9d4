// mx_layer_api.cpp -- the C ABI (include/mx.h) of the operators between a layer's
// products: the choice of experts, the norms around a block.  Validation is pure
// host code and runs before any device call.
#include <hip/hip_runtime.h>

#include <cmath>

#include "mx_host.h"

namespace {

using namespace mx;

bool ld_bad(int64_t ld, int64_t cols) { return ld < cols || ld > kMaxLd; }
bool aligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
hipStream_t hip(mx_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

mx_status mx_moe_route(int64_t E, int64_t T, int64_t topk, int type, const void *logits,
                       int64_t ldl, int score, const float *bias, int64_t groups,
                       int64_t topk_groups, int group_best, int renorm, float scale,
                       int32_t *topk_ids, float *topk_weights, mx_stream_t stream) {
    if (type != FLOAT_BF16 && type != FLOAT_F32) return MX_ERR_UNSUPPORTED;
    if (score != SCORE_SOFTMAX && score != SCORE_SIGMOID) return MX_ERR_UNSUPPORTED;
    if ((group_best != 1 && group_best != 2) || (renorm != 0 && renorm != 1))
        return MX_ERR_UNSUPPORTED;
    if (E < 1 || E > kRouteMaxExperts || T < 1 || topk < 1 || topk > E || topk > kRouteMaxTopk ||
        T > kMaxRows / topk || ld_bad(ldl, E) || !std::isfinite(scale))
        return MX_ERR_SHAPE;
    if (groups < 1 || groups > kRouteMaxGroups || E % groups != 0 || topk_groups < 1 ||
        topk_groups > groups || topk > topk_groups * (E / groups) || group_best > E / groups)
        return MX_ERR_SHAPE;
    // two logits without a bias have no sum of scores
    if (group_best == 2 && !bias) return MX_ERR_UNSUPPORTED;
    if (!logits || !topk_ids || !topk_weights) return MX_ERR_NULL;
    if (!(type == FLOAT_BF16 ? aligned2(logits) : aligned4(logits)) || (bias && !aligned4(bias)) ||
        !aligned4(topk_ids) || !aligned4(topk_weights))
        return MX_ERR_ALIGN;
    const Span in{logits, T, ldl, E, type == FLOAT_BF16 ? 2 : 4}, sb{bias, 1, 0, E, 4};
    const Span si{topk_ids, 1, 0, T * topk, 4}, sw{topk_weights, 1, 0, T * topk, 4};
    if (overlap(si, in) || overlap(si, sb) || overlap(sw, in) || overlap(sw, sb) || overlap(si, sw))
        return MX_ERR_UNSUPPORTED;
    const mx_status st = device_ok();
    if (st != MX_OK) return st;
    RouteArgs a{};
    a.T = T;
    a.E = (int)E;
    a.topk = (int)topk;
    a.logits = logits;
    a.ldl = ldl;
    a.bias = bias;
    a.score = score;
    a.groups = (int)groups;
    a.per_group = (int)(E / groups);
    // every group kept: none of them matters
    if (topk_groups == groups) a.groups = 1;
    a.topk_groups = (int)topk_groups;
    a.group_best = group_best;
    a.group_mul = (int)(((1 << 20) + E / groups - 1) / (E / groups));
    a.renorm = renorm;
    a.scale = scale;
    a.ids = topk_ids;
    a.weights = topk_weights;
    log_dispatch("moe_route: route_kernel, %s logits, %s%s, %lld of %lld groups; E=%lld T=%lld "
                 "topk=%lld",
                 type == FLOAT_BF16 ? "bf16" : "fp32",
                 score == SCORE_SOFTMAX ? "softmax" : "sigmoid", bias ? " with bias" : "",
                 (long long)topk_groups, (long long)groups, (long long)E, (long long)T,
                 (long long)topk);
    return launched(launch_moe_route(a, type, hip(stream)));
}

mx_status mx_block_norm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *post_weight,
                        const void *gate, int64_t gates, int64_t ldg, const int32_t *gate_ids,
                        int stream_type, const void *residual, int64_t ldr, float alpha,
                        const void *weight, float offset, float eps, int act, int rule, void *sum,
                        int64_t lds, void *y, int64_t ldy, void *xq, int64_t ldq, void *xcodes,
                        int64_t ldc, mx_stream_t stream) {
    if (act != ACT_BF16 && act != ACT_MXFP8 && act != ACT_MXFP8_T16) return MX_ERR_UNSUPPORTED;
    if (rule != RULE_OCP && rule != RULE_CEIL448) return MX_ERR_UNSUPPORTED;
    if (stream_type != FLOAT_BF16 && stream_type != FLOAT_F32) return MX_ERR_UNSUPPORTED;
    if (!weight && act != ACT_BF16) return MX_ERR_UNSUPPORTED;     // no norm to quantize
    const int64_t size = stream_type == FLOAT_F32 ? 4 : 2;
    if (M < 1 || M > kMaxRows || K < 32 || K % 32 != 0 || K > kNormMaxK || !(eps >= 0.0f) ||
        !std::isfinite(alpha) || !std::isfinite(offset))
        return MX_ERR_SHAPE;
    if (!x) return MX_ERR_NULL;
    if (weight ? (act == ACT_BF16 ? !y : (!xq || !xcodes)) : !sum) return MX_ERR_NULL;
    if (!weight && y) return MX_ERR_UNSUPPORTED;
    if (ld_bad(ldx, K) || (residual && ld_bad(ldr, K)) || (sum && ld_bad(lds, K)) ||
        (y && ld_bad(ldy, K)))
        return MX_ERR_SHAPE;
    if (gate && (gates < 1 || gates > kMaxRows || ld_bad(ldg, K))) return MX_ERR_SHAPE;
    if (act == ACT_MXFP8 && (ld_bad(ldq, K) || ld_bad(ldc, K / 32))) return MX_ERR_SHAPE;
    // 16-byte pieces of every row
    const int64_t per = 16 / size;
    if (!aligned16(x) || ldx % 8 != 0 || (post_weight && !aligned16(post_weight)) ||
        (weight && !aligned16(weight)) || (gate && (!aligned16(gate) || ldg % 8 != 0)) ||
        (gate && gate_ids && !aligned4(gate_ids)) ||
        (residual && (!aligned16(residual) || ldr % per != 0)) ||
        (sum && (!aligned16(sum) || lds % per != 0)) || (y && (!aligned16(y) || ldy % 8 != 0)))
        return MX_ERR_ALIGN;
    if (act != ACT_BF16 && (!aligned16(xq) || (act == ACT_MXFP8 && ldq % 16 != 0) ||
                            (act == ACT_MXFP8_T16 && !aligned16(xcodes))))
        return MX_ERR_ALIGN;
    const Span sx{x, M, ldx, K, 2}, sr{residual, M, ldr, K, size};
    const Span ss{sum, M, lds, K, size}, sy{y, M, ldy, K, 2};
    const Span ins[] = {{post_weight, 1, K, K, 2},
                        {weight, 1, K, K, 2},
                        {gate, gates, ldg, K, 2},
                        {gate ? gate_ids : nullptr, 1, 0, M, 4}};
    Span sq{nullptr, 1, 0, 0, 1}, sc{nullptr, 1, 0, 0, 1};
    if (act == ACT_MXFP8) {
        sq = {xq, M, ldq, K, 1};
        sc = {xcodes, M, ldc, K / 32, 1};
    } else if (act == ACT_MXFP8_T16) {
        sq = {xq, 1, 0, act_t16_data_bytes(M, K), 1};
        sc = {xcodes, 1, 0, act_codes_t16_bytes(M, K), 1};
    }
    // sum and y may stand on an input of their own element size
    if (!apart_or_same(ss, sr) || !apart_or_same(sy, sx) || overlap(ss, sy) ||
        (size == 2 ? !apart_or_same(ss, sx) || !apart_or_same(sy, sr)
                   : overlap(ss, sx) || overlap(sy, sr)))
        return MX_ERR_UNSUPPORTED;
    for (const Span &out : {ss, sy, sq, sc})
        for (const Span &in : ins)
            if (overlap(out, in)) return MX_ERR_UNSUPPORTED;
    for (const Span &out : {sq, sc})
        if (overlap(out, sx) || overlap(out, sr) || overlap(out, ss) || overlap(out, sy))
            return MX_ERR_UNSUPPORTED;
    if (overlap(sq, sc)) return MX_ERR_UNSUPPORTED;
    const mx_status st = device_ok();
    if (st != MX_OK) return st;
    BlockNormArgs a{};
    a.M = M;
    a.K = K;
    a.x = static_cast<const uint16_t *>(x);
    a.ldx = ldx;
    a.post = static_cast<const uint16_t *>(post_weight);
    a.gate = static_cast<const uint16_t *>(gate);
    a.gates = gates;
    a.ldg = ldg;
    a.gate_ids = gate_ids;
    a.res = residual;
    a.ldr = ldr;
    a.alpha = alpha;
    a.weight = static_cast<const uint16_t *>(weight);
    a.offset = offset;
    a.eps = eps;
    a.sum = sum;
    a.lds = lds;
    a.y = static_cast<uint16_t *>(y);
    a.ldy = ldy;
    a.xq = static_cast<uint8_t *>(xq);
    a.ldq = ldq;
    a.xcodes = static_cast<uint8_t *>(xcodes);
    a.ldc = ldc;
    a.rule = rule;
    log_dispatch("block_norm: block_norm_kernel,%s%s %s stream, %s output (rule %d); M=%lld K=%lld",
                 post_weight ? " post norm," : "", gate ? " gate," : "",
                 stream_type == FLOAT_F32 ? "fp32" : "bf16",
                 !weight             ? "no"
                 : act == ACT_BF16   ? "bf16"
                 : act == ACT_MXFP8  ? "row-major MXFP8"
                                     : "T16",
                 rule, (long long)M, (long long)K);
    return launched(launch_block_norm(a, stream_type, act, hip(stream)));
}

}  // extern "C"
