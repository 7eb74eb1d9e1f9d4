// mx_router.hip -- the choice of experts from router logits.
//
//   s = softmax(x) or sigmoid(x) in fp32;  c = s + bias, or x without a bias
//   a group's score: the sum of its one or two largest c; the best groups are kept
//   ids: the topk largest c of the kept groups, equal ones by lower index
//   w = scale * s of the chosen, with renorm over their sum
// Without a bias the choice goes by the logits, whose order is the scores' without
// their rounding: no score is needed but the chosen ones'.  With a bias each score is
// formed in 64 bits and rounded once to fp32: the choice is then a function of the
// inputs alone (fp32 functions of another last place would order near-equal sums
// otherwise), and equal scores tie.
//
// LPT lanes share a token (64 / LPT tokens a wavefront); lane i holds the experts
// 4 (i + LPT c) + d, d < 4, c < C, one 16-byte load (bf16: 8) for each c.  A choice is a
// maximum over (c, lower index first): the sortable 32 bits of c above 1023 - expert
// make a 62-bit number, which read as a double is positive and finite, so one
// v_max_f64 orders both.  topk rounds: each lane's maximum, DPP steps over the
// token's lanes, the winner struck out.  Groups are scored from LDS, a lane a group,
// starting at its own place in the group so that the lanes meet different banks.
// Wavefronts are independent; LDS serves one wavefront's exchange (operations of a
// wavefront complete in order).
//
// Sums of exponentials are added as chunks of four experts, then over the chunk
// number's bits in an order that is the same in every form: a token's results do not
// depend on the other tokens or their number.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_lanes.h"

#include <cfloat>

namespace mx {

constexpr int kRouteWaves = 4;             // independent wavefronts a workgroup

// a sum over the C chunks of a lane, in the order of their number's bits
template <int C, class T>
__device__ inline T chunk_sum(const T (&v)[C]) {
    if constexpr (C == 4) return (v[0] + v[1]) + (v[2] + v[3]);
    else if constexpr (C == 2) return v[0] + v[1];
    else return v[0];
}

template <int LPT, int C, bool BF16, bool VEC, bool BIAS>
__global__ void __launch_bounds__(64 * kRouteWaves) route_kernel(RouteArgs p) {
    constexpr int TOK = 64 / LPT;                         // tokens of a wavefront
    constexpr int EP = 4 * LPT * C;                       // experts with room
    __shared__ float xs_[kRouteWaves][TOK][EP];           // logits; -inf: masked
    __shared__ float cs_[kRouteWaves][TOK][EP];           // c, when there are groups
    __shared__ float gs_[kRouteWaves][TOK][kRouteMaxGroups];
    __shared__ int out_[kRouteWaves][TOK][kRouteMaxTopk];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int tok = lane / LPT, i = lane % LPT;
    const int E = p.E;
    const int64_t t = ((int64_t)blockIdx.x * kRouteWaves + wave) * TOK + tok;
    const bool live = t < p.T;
    float *xs = xs_[wave][tok], *cs = cs_[wave][tok], *gs = gs_[wave][tok];
    int *out = out_[wave][tok];

    // ---- logits: masked ones (and what lies past E) are -inf ----
    float x[C][4];
    const int64_t row = (live ? t : 0) * p.ldl;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = 4 * (i + LPT * c);
        if constexpr (BF16) {
            const uint16_t *src = static_cast<const uint16_t *>(p.logits) + row + e0;
            if constexpr (VEC) {
                v2u v = {0xFF80FF80u, 0xFF80FF80u};
                if (live && e0 < E) v = *reinterpret_cast<const v2u *>(src);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    x[c][d] = __uint_as_float(d % 2 ? v[d / 2] & 0xFFFF0000u : v[d / 2] << 16);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    x[c][d] = live && e0 + d < E ? bf16_to_f32(src[d]) : -INFINITY;
            }
        } else {
            const float *src = static_cast<const float *>(p.logits) + row + e0;
            if constexpr (VEC) {
                v4f v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (live && e0 < E) v = *reinterpret_cast<const v4f *>(src);
#pragma unroll
                for (int d = 0; d < 4; ++d) x[c][d] = v[d];
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) x[c][d] = live && e0 + d < E ? src[d] : -INFINITY;
            }
        }
    }
    float b[C][4];
    if constexpr (BIAS) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int e = 4 * (i + LPT * c) + d;
                b[c][d] = e < E ? p.bias[e] : -INFINITY;
            }
    }
    // NaN is masked too, +inf counts as the largest number
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            x[c][d] = x[c][d] > -INFINITY ? __builtin_fminf(x[c][d], FLT_MAX) : -INFINITY;
            top = __builtin_fmaxf(top, x[c][d]);
            xs[4 * (i + LPT * c) + d] = x[c][d];
        }

    // ---- the largest logit and the sum of exponentials (softmax) ----
    float sum32 = 1.0f;
    double sum64 = 1.0;
    if (p.score == SCORE_SOFTMAX) {
        top = lanes_max<LPT>(top);
        if (!(top > -INFINITY)) top = 0.0f;               // nothing is left: every s is 0
        if constexpr (BIAS) {
            double part[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                double v[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = exp((double)x[c][d] - (double)top);
                part[c] = (v[0] + v[1]) + (v[2] + v[3]);
            }
            sum64 = over_lanes64<LPT>(chunk_sum(part), [](double a, double b2) { return a + b2; });
        } else {
            float part[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = expf(x[c][d] - top);
                part[c] = (v[0] + v[1]) + (v[2] + v[3]);
            }
            sum32 = lanes_sum<LPT>(chunk_sum(part));
        }
    }
    auto score64 = [&](float v) -> float {
        if (p.score == SCORE_SIGMOID) return (float)(1.0 / (1.0 + exp(-(double)v)));
        return (float)(exp((double)v - (double)top) / sum64);
    };
    auto score32 = [&](float v) -> float {
        if (p.score == SCORE_SIGMOID) {
            const float e = expf(-__builtin_fabsf(v));    // no overflow: tiny scores stay
            return (v < 0.0f ? e : 1.0f) / (1.0f + e);
        }
        return expf(v - top) / sum32;
    };

    // ---- what the choice goes by ----
    float key[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            float k = x[c][d];
            if constexpr (BIAS) {
                const bool in = k > -INFINITY && b[c][d] > -INFINITY;
                k = in ? __builtin_fminf(score64(k) + b[c][d], FLT_MAX) : -INFINITY;
            }
            key[c][d] = k + 0.0f;                         // -0 is 0
        }

    // ---- groups ----
    if (p.groups > 1) {
        const int G = p.groups, n = p.per_group;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) cs[4 * (i + LPT * c) + d] = key[c][d];
        wave_order();
        for (int g = i; g < G; g += LPT) {
            float m1 = -INFINITY, m2 = -INFINITY;
            int j = g % n;
            for (int k = 0; k < n; ++k) {
                const float v = cs[g * n + j];
                m2 = __builtin_fmaxf(m2, __builtin_fminf(m1, v));
                m1 = __builtin_fmaxf(m1, v);
                j = j + 1 == n ? 0 : j + 1;
            }
            gs[g] = p.group_best == 2 ? m1 + m2 : m1;
        }
        wave_order();
        // a group is kept when fewer than topk_groups are ahead of it
        uint64_t kept = 0;
        for (int base = 0; base < G; base += LPT) {
            const int g = base + i;
            const float v = g < G ? gs[g] : 0.0f;
            int ahead = 0;
            for (int h = 0; h < G; ++h) {
                const float u = gs[h];
                ahead += u > v || (u == v && h < g) ? 1 : 0;
            }
            const uint64_t in = __ballot(g < G && ahead < p.topk_groups) >> (tok * LPT);
            kept |= (LPT == 64 ? in : in & ((1ull << (LPT % 64)) - 1ull)) << base;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int e = 4 * (i + LPT * c) + d;
                const uint32_t g = (uint32_t)e * (uint32_t)p.group_mul >> 20;   // e / n
                if (!(kept >> (g & 63u) & 1u)) key[c][d] = -INFINITY;
            }
    }

    // ---- topk rounds ----
    double best[C][4];                                    // 0: not to be chosen
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t u = __float_as_uint(key[c][d]);
            const uint32_t s = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
            const uint32_t e = (uint32_t)(4 * (i + LPT * c) + d);
            const uint64_t v = (uint64_t)s << 30 | (1023u - e);
            best[c][d] = __builtin_bit_cast(double, key[c][d] > -INFINITY ? v : uint64_t(0));
        }
    for (int r = 0; r < p.topk; ++r) {
        double m = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) m = __builtin_fmax(m, best[c][d]);
        m = over_lanes64<LPT>(m, [](double a, double b2) { return __builtin_fmax(a, b2); });
        const uint64_t won = __builtin_bit_cast(uint64_t, m);
        if (i == 0) out[r] = won ? 1023 - (int)(won & 1023u) : -1;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint64_t v = __builtin_bit_cast(uint64_t, best[c][d]);
                best[c][d] = __builtin_bit_cast(double, v == won ? uint64_t(0) : v);
            }
    }
    wave_order();

    // ---- weights: lane r of the token finishes choice r (and r + LPT, ..) ----
    float *w = gs;                                        // the groups' scores are done with
    if (live)
        for (int r = i; r < p.topk; r += LPT) {
            const int e = out[r];
            float s = 0.0f;
            if (e >= 0) s = BIAS ? score64(xs[e]) : score32(xs[e]);
            w[r] = s;
        }
    wave_order();
    float sum = 1.0f;
    if (p.renorm) {
        sum = 0.0f;
        for (int r = 0; r < p.topk; ++r) sum += w[r];     // in order: the same in every form
    }
    if (live)
        for (int r = i; r < p.topk; r += LPT) {
            p.ids[t * p.topk + r] = out[r];
            p.weights[t * p.topk + r] = sum > 0.0f ? p.scale * (w[r] / sum) : 0.0f;
        }
}

template <int LPT, int C, bool BF16, bool VEC>
static hipError_t launch_bias(const RouteArgs &a, hipStream_t st) {
    const int64_t per = kRouteWaves * (64 / LPT);
    const dim3 grid((unsigned)((a.T + per - 1) / per)), block(64 * kRouteWaves);
    if (a.bias) hipLaunchKernelGGL((route_kernel<LPT, C, BF16, VEC, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((route_kernel<LPT, C, BF16, VEC, false>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <int LPT, int C>
static hipError_t launch_type(const RouteArgs &a, int type, hipStream_t st) {
    const int size = type == FLOAT_BF16 ? 2 : 4;
    // four experts at once where every row starts on a multiple of their size
    const bool vec = a.E % 4 == 0 && a.ldl % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(a.logits) % (4 * size) == 0;
    if (type == FLOAT_BF16)
        return vec ? launch_bias<LPT, C, true, true>(a, st) : launch_bias<LPT, C, true, false>(a, st);
    return vec ? launch_bias<LPT, C, false, true>(a, st) : launch_bias<LPT, C, false, false>(a, st);
}

// Few tokens: a wavefront each, the shortest rounds.  Many: as few lanes a token as
// hold its experts, so that a round serves several tokens.
hipError_t launch_moe_route(const RouteArgs &a, int type, hipStream_t st) {
    if (a.E > 512) return launch_type<64, 4>(a, type, st);
    if (a.E > 256) return launch_type<32, 4>(a, type, st);
    if (a.T <= 1024) return launch_type<64, 1>(a, type, st);
    if (a.E > 128) return launch_type<16, 4>(a, type, st);
    if (a.E > 64) return launch_type<16, 2>(a, type, st);
    if (a.E > 32) return launch_type<16, 1>(a, type, st);
    return launch_type<8, 1>(a, type, st);
}

}  // namespace mx
