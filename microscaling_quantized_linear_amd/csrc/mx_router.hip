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
// 4 (i + LPT c) + d, d < 4, c < C, one 16-byte load (bf16: 8) for each c.  c is held as a
// 32-bit number of the same order.  Choosing:
//   a bound that more than topk experts reach: where topk < LPT <= 16, the smallest
//     of the lanes' maxima that fewer than topk + 1 lanes' maxima exceed (each lane counts
//     them by DPP rotations); else, and where too few lanes hold experts of a kept group,
//     the topk + 1 largest distinct numbers one by one (the differences to the last one
//     modulo 2^32 put what is not below it last);
//   the experts at or above it, some more than topk, into a list in LDS;
//   a lane an entry counts the entries ahead of it: the larger, and the equal of a
//     lower expert.
// With a bias c comes from fast fp32 scores first: groups and the list go by them, the
// list with the fast scores' error bound added to it, and the list's entries are then
// formed in 64 bits.  Where a token's last kept and first dropped group are nearer than
// the error bound, the scores that may be among their groups' best are formed in 64 bits
// first (every score of the wavefront's tokens: 15.0 us instead of 14.0 for the call
// below, whose end waits for the few wavefronts that this happens to).  The result is
// the exact choice either way.  A list that overflows (many equal numbers)
// gives way to rounds of one expert each.
// Bound: the vector instructions, all tokens in one round of the chip's wavefronts.  E
// 256, T 16384, top 8 of 4 of 8 groups: 13.2-14.0 us by box (18 MB, 3.8 us of a copy's
// time); 1170 vector instructions a wavefront, four wavefronts a SIMD, which issues them
// for 19,300 of the 22,900 cycles that a wavefront lives; four times the tokens take 37
// us.  With 64-bit scores for all and a maximum a round 22.3.  A decode step's 16 tokens:
// 4.0 us, with a bias and groups 5.1: launch and two trips to memory.
// More than 256 experts take the bound one by one, 32 or 64 lanes a token: E 384, top 8,
// T 4096 / 16384 5.4 / 12.8 us (with a bias 6.2 / 15.7), E 512, top 10 5.8 / 14.3.  A list
// that cannot hold topk + 1 and what is near them gives way to the rounds: topk 64 always,
// 63 nearly so (E 256, T 4096 31 and 25 us, with a bias 36 and 35; topk 32 9.6 and 10.8).
// Groups of 4, 8, .. 64 experts are scored in registers, over the lanes that hold them
// (E 64, T 16384, 8 groups: 8.0 us, the other form 8.4), others from LDS, a lane a group, starting at its own place
// in the group so that the lanes meet different banks.  Wavefronts are independent; LDS serves one
// wavefront's exchange (operations of a wavefront complete in order).
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
constexpr int kRouteList = 64;             // experts that are ranked against each other

// a sum over the C chunks of a lane, in the order of their number's bits
template <int C, class T>
__device__ inline T chunk_sum(const T (&v)[C]) {
    if constexpr (C == 8)                                 // choices of 8-lane tokens: bits 4, 5, 3
        return ((v[0] + v[2]) + (v[4] + v[6])) + ((v[1] + v[3]) + (v[5] + v[7]));
    else if constexpr (C == 4) return (v[0] + v[1]) + (v[2] + v[3]);
    else if constexpr (C == 2) return v[0] + v[1];
    else return v[0];
}

// 2^x by v_exp_f32 (within a last place)
__device__ inline float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float kLog2e = 1.4426950408889634f;

// e^d for d <= 0, within 2^-46 of itself: 2^t by its series about t's nearest whole
// number, (ln 2 / 2)^12 / 12! being 2^-47 (the general function takes twice as long).
// -inf gives 0, as does what lies below the smallest double.
__device__ inline double exp64(double d) {
    const double t = __builtin_fmax(d * 1.4426950408889634, -1100.0);
    const double n = __builtin_rint(t), r = (t - n) * 0.6931471805599453;
    double v = 1.0 / 39916800.0;
    v = __builtin_fma(v, r, 1.0 / 3628800.0);
    v = __builtin_fma(v, r, 1.0 / 362880.0);
    v = __builtin_fma(v, r, 1.0 / 40320.0);
    v = __builtin_fma(v, r, 1.0 / 5040.0);
    v = __builtin_fma(v, r, 1.0 / 720.0);
    v = __builtin_fma(v, r, 1.0 / 120.0);
    v = __builtin_fma(v, r, 1.0 / 24.0);
    v = __builtin_fma(v, r, 1.0 / 6.0);
    v = __builtin_fma(v, r, 0.5);
    v = __builtin_fma(v, r, 1.0);
    v = __builtin_fma(v, r, 1.0);
    return __builtin_amdgcn_ldexp(v, (int)n);
}
// 1 / (1 + e^-v), to 2^-44: one Newton step on an fp32 reciprocal
__device__ inline double sigmoid64(double v) {
    const double e = exp64(-__builtin_fabs(v)), a = 1.0 + e;
    const double y = (double)__builtin_amdgcn_rcpf((float)a);
    const double q = __builtin_fma(__builtin_fma(-a, y, 1.0), y, y);
    return v < 0.0 ? e * q : q;
}

// four workgroups a compute unit; three of 8-lane tokens, whose LDS takes 45 KB
template <int LPT, int C, bool BF16, bool VEC, bool BIAS>
__global__ void __launch_bounds__(64 * kRouteWaves, LPT == 8 ? 3 : 4) route_kernel(RouteArgs p) {
    constexpr int TOK = 64 / LPT;                         // tokens of a wavefront
    constexpr int EP = 4 * LPT * C;                       // experts with room
    constexpr uint32_t kNone = 0x007FFFFFu;               // the number of -inf
    __shared__ __attribute__((aligned(16))) float cs_[kRouteWaves][TOK][EP];   // c, -inf: masked
    // the groups' scores, then the list: a number above ~expert
    __shared__ __attribute__((aligned(16))) uint64_t list_[kRouteWaves][TOK][kRouteList];
    __shared__ uint16_t es_[kRouteWaves][TOK][kRouteList];
    __shared__ uint16_t out_[kRouteWaves][TOK][kRouteMaxTopk];
    __shared__ float ss_[kRouteWaves][TOK][kRouteList];   // the list's scores
    __shared__ float ws_[kRouteWaves][TOK][kRouteMaxTopk];
    static_assert(2 * kRouteList >= kRouteMaxGroups && kRouteList % 16 == 0, "room for either");
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int tok = lane / LPT, i = lane % LPT;
    const int E = p.E;
    const int64_t t = ((int64_t)blockIdx.x * kRouteWaves + wave) * TOK + tok;
    const bool live = t < p.T;
    float *cs = cs_[wave][tok], *gs = reinterpret_cast<float *>(list_[wave][tok]);
    uint64_t *list = list_[wave][tok];
    uint16_t *es = es_[wave][tok], *out = out_[wave][tok];
    float *ss = ss_[wave][tok], *w = ws_[wave][tok];
    const int64_t row = (live ? t : 0) * p.ldl;
    const bool softmax = p.score == SCORE_SOFTMAX;
    // NaN is masked too, +inf the largest number
    auto clean = [](float v) -> float {
        return __builtin_fminf(__builtin_fmaxf(v, -INFINITY), FLT_MAX);
    };
    auto logit = [&](int e) -> float {
        return clean(BF16 ? bf16_to_f32(static_cast<const uint16_t *>(p.logits)[row + e])
                          : static_cast<const float *>(p.logits)[row + e]);
    };

    // ---- logits: masked ones (and what lies past E) are -inf ----
    float x[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = 4 * (i + LPT * c);
        if constexpr (VEC && BF16) {
            const uint16_t *src = static_cast<const uint16_t *>(p.logits) + row + e0;
            v2u v = {0xFF80FF80u, 0xFF80FF80u};
            if (live && e0 < E) v = *reinterpret_cast<const v2u *>(src);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                x[c][d] = clean(__uint_as_float(d % 2 ? v[d / 2] & 0xFFFF0000u : v[d / 2] << 16));
        } else if constexpr (VEC) {
            const float *src = static_cast<const float *>(p.logits) + row + e0;
            v4f v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (live && e0 < E) v = *reinterpret_cast<const v4f *>(src);
#pragma unroll
            for (int d = 0; d < 4; ++d) x[c][d] = clean(v[d]);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) x[c][d] = live && e0 + d < E ? logit(e0 + d) : -INFINITY;
        }
    }

    // ---- the largest logit and the sum of exponentials (softmax) ----
    float top = 0.0f, inv = 1.0f;
    if (softmax) {
        top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) top = __builtin_fmaxf(top, x[c][d]);
        top = lanes_max<LPT>(top);
        if (!(top > -INFINITY)) top = 0.0f;               // nothing is left: every s is 0
        float part[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = exp2_hw((x[c][d] - top) * kLog2e);
            part[c] = (v[0] + v[1]) + (v[2] + v[3]);
        }
        inv = 1.0f / lanes_sum<LPT>(chunk_sum(part));
    }
    double sum64 = 1.0;
    if (BIAS && softmax) {
        double part[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            double v[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = exp64((double)x[c][d] - (double)top);
            part[c] = (v[0] + v[1]) + (v[2] + v[3]);
        }
        sum64 = over_lanes64<LPT>(chunk_sum(part), [](double a, double b) { return a + b; });
    }
    // the score of a logit, -inf's being 0
    auto score = [&](float v) -> float {
        if constexpr (BIAS)
            return (float)(softmax ? exp64((double)v - (double)top) / sum64 : sigmoid64((double)v));
        if (softmax) return expf(v - top) * inv;
        const float u = expf(-__builtin_fabsf(v));        // no overflow: tiny scores stay
        return (v < 0.0f ? u : 1.0f) / (1.0f + u);
    };

    // ---- what the choice goes by ----
    float f[C][4];
    if constexpr (BIAS) {
        if (softmax) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d) f[c][d] = exp2_hw((x[c][d] - top) * kLog2e) * inv;
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    f[c][d] = __builtin_amdgcn_rcpf(1.0f + exp2_hw(-kLog2e * x[c][d]));
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e0 = 4 * (i + LPT * c);
            v4f b = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (VEC) {
                if (e0 < E) b = *reinterpret_cast<const v4f *>(p.bias + e0);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) b[d] = e0 + d < E ? p.bias[e0 + d] : 0.0f;
            }
#pragma unroll
            for (int d = 0; d < 4; ++d)
                f[c][d] = x[c][d] > -INFINITY ? clean(f[c][d] + b[d]) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) f[c][d] = x[c][d] + 0.0f;   // -0 is 0
    }
    // The fast scores' distance from the exact ones: sigmoid s (1 - s) (|x| 2^-22 +
    // 2^-23) <= 2^-24, the reciprocal and the sum's roundings 2^-22; softmax d e^-d
    // 2^-22 and the sum's 2^-21 of the largest score: both doubled, and two for a
    // difference.  Adding the bias rounds to |c| 2^-24 on either side.
    const float eps = softmax ? 0x1p-18f * inv : 0x1p-20f;
    auto error = [&](float c) -> float { return __builtin_fmaf(__builtin_fabsf(c), 0x1p-22f, eps); };
    // a number of c's order
    auto number = [](float c) -> uint32_t {
        const uint32_t u = __float_as_uint(c);
        return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    };
    auto value = [](uint32_t s) -> float {
        return __uint_as_float(s & 0x80000000u ? s ^ 0x80000000u : ~s);
    };

    // this lane's experts (bit 4 c + d) that may be among their groups' best
    uint32_t near = ~0u;
    // the groups that are kept, as bits of g; `doubt` where the fast scores do not tell
    auto keep_groups = [&](bool &doubt) -> uint64_t {
        const int G = p.groups, n = p.per_group, span = n / 4;
        if (n % 4 == 0 && (span & (span - 1)) == 0 && span <= (LPT < 16 ? LPT : 16)) {
            // the group's chunks lie in `span` neighbouring lanes (uniform)
            float m1[C], m2[C];                           // the two largest
            auto join = [&](int c, float u1, float u2) {
                m2[c] = __builtin_fmaxf(__builtin_fminf(m1[c], u1), __builtin_fmaxf(m2[c], u2));
                m1[c] = __builtin_fmaxf(m1[c], u1);
            };
#pragma unroll
            for (int c = 0; c < C; ++c) {
                m1[c] = __builtin_fmaxf(f[c][0], f[c][1]);
                m2[c] = __builtin_fminf(f[c][0], f[c][1]);
                join(c, __builtin_fmaxf(f[c][2], f[c][3]), __builtin_fminf(f[c][2], f[c][3]));
            }
            auto meet = [&](auto ctrl) {
                constexpr int CTRL = decltype(ctrl)::value;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    join(c, __uint_as_float(dpp<CTRL>(__float_as_uint(m1[c]))),
                         __uint_as_float(dpp<CTRL>(__float_as_uint(m2[c]))));
            };
            if (span > 1) meet(std::integral_constant<int, kSwap1>{});
            if (span > 2) meet(std::integral_constant<int, kSwap2>{});
            if (span > 4) meet(std::integral_constant<int, kHalfMirror>{});
            if (span > 8) meet(std::integral_constant<int, kRotate8>{});
            if constexpr (BIAS) {
                // the last of a group's best is at least its fast score less the error,
                // and an expert's fast score at least its own less as much
                near = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float last = p.group_best == 2 ? m2[c] : m1[c];
                    const float least = last - 3.0f * error(last);
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        near |= f[c][d] > -INFINITY && f[c][d] >= least ? 1u << (4 * c + d) : 0u;
                }
            }
            const int shift = __ffs(span) - 1;
            if ((i & (span - 1)) == 0)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int g = (i + LPT * c) >> shift;
                    if (g < G) gs[g] = p.group_best == 2 ? m1[c] + m2[c] : m1[c];
                }
        } else
        for (int g = i; g < G; g += LPT) {
            float m1 = -INFINITY, m2 = -INFINITY;         // the two largest so far
            auto take = [&](float v) {
                m2 = __builtin_amdgcn_fmed3f(m1, m2, v);
                m1 = __builtin_fmaxf(m1, v);
            };
            if (n % 4 == 0) {
                const int quads = n / 4;
                int j = g % quads;
                for (int k = 0; k < quads; ++k) {
                    const v4f v = *reinterpret_cast<const v4f *>(cs + g * n + 4 * j);
                    take(v[0]);
                    take(v[1]);
                    take(v[2]);
                    take(v[3]);
                    j = j + 1 == quads ? 0 : j + 1;
                }
            } else {
                int j = g % n;
                for (int k = 0; k < n; ++k) {
                    take(cs[g * n + j]);
                    j = j + 1 == n ? 0 : j + 1;
                }
            }
            gs[g] = p.group_best == 2 ? m1 + m2 : m1;
        }
        wave_order();
        // kept when fewer than topk_groups are ahead
        uint64_t kept = 0;
        float least = INFINITY, most = -INFINITY;         // of the kept, of the dropped
        for (int base = 0; base < G; base += LPT) {
            const int g = base + i;
            const float v = g < G ? gs[g] : 0.0f;
            int ahead = 0;
#pragma unroll 8
            for (int h = 0; h < G; ++h) {
                const float u = gs[h];
                ahead += u > v || (u == v && h < g) ? 1 : 0;
            }
            const bool in = g < G && ahead < p.topk_groups;
            if (in) least = __builtin_fminf(least, v);
            else if (g < G) most = __builtin_fmaxf(most, v);
            const uint64_t mine = __ballot(in) >> (tok * LPT);
            kept |= (LPT == 64 ? mine : mine & ((1ull << (LPT % 64)) - 1ull)) << base;
        }
        if constexpr (BIAS) {
            least = -lanes_max<LPT>(-least);
            most = lanes_max<LPT>(most);
            // (where nothing dropped has a score there is no doubt)
            doubt = most > -INFINITY && !(least - most > 2.0f * (error(least) + error(most)));
        }
        wave_order();
        return kept;
    };
    // all ones where expert e's group is kept
    auto kept_mask = [&](uint64_t kept, int e) -> uint32_t {
        const uint32_t g = __umul24((uint32_t)e, (uint32_t)p.group_mul) >> 20;   // e / n
        const uint32_t half = g & 32u ? (uint32_t)(kept >> 32) : (uint32_t)kept;
        return 0u - (half >> (g & 31u) & 1u);
    };
    uint32_t key[C][4];
    auto keys = [&](bool &doubt) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            *reinterpret_cast<v4f *>(cs + 4 * (i + LPT * c)) = v4f{f[c][0], f[c][1], f[c][2], f[c][3]};
#pragma unroll
            for (int d = 0; d < 4; ++d) key[c][d] = number(f[c][d]);
        }
        wave_order();
        if (p.groups > 1) {
            const uint64_t kept = keep_groups(doubt);
            if (p.per_group % 4 == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t m = kept_mask(kept, 4 * (i + LPT * c));
#pragma unroll
                    for (int d = 0; d < 4; ++d) key[c][d] &= m;
                }
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int d = 0; d < 4; ++d) key[c][d] &= kept_mask(kept, 4 * (i + LPT * c) + d);
            }
        }
    };
    auto keep_logits = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c)
            *reinterpret_cast<v4f *>(cs + 4 * (i + LPT * c)) = v4f{x[c][0], x[c][1], x[c][2], x[c][3]};
        wave_order();
    };
    // c with its score from 64 bits, for the experts `which` of this lane
    auto exact = [&](const uint32_t which) {
        keep_logits();
        uint32_t left = which;
        while (__ballot(left != 0u)) {
            if (left) {
                const int k = __ffs((int)left) - 1, e = 4 * (i + LPT * (k / 4)) + k % 4;
                left &= left - 1u;
                const float v = cs[e], b = e < E ? p.bias[e] : 0.0f;
                cs[e] = v > -INFINITY ? clean(score(v) + b) : -INFINITY;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const v4f v = *reinterpret_cast<const v4f *>(cs + 4 * (i + LPT * c));
#pragma unroll
            for (int d = 0; d < 4; ++d) f[c][d] = which >> (4 * c + d) & 1u ? v[d] : f[c][d];
        }
    };
    constexpr uint32_t kEvery = (1u << (4 * C)) - 1u;
    static_assert(C <= 4, "a lane's experts are bits of a word");
    bool doubt = false;
    keys(doubt);
    if constexpr (BIAS)
        if (__ballot(doubt && live)) {
            exact(doubt ? near & kEvery : 0u);
            keys(doubt);
        }
    if constexpr (BIAS) keep_logits();                    // without a bias they stand there

    // ---- a bound that more than topk experts reach, or all that are left ----
    auto more = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    uint32_t mine = 0;                                    // this lane's experts that reach it
    int count = 0, behind = 0, n = 0;                     // theirs, with the lanes before, in all
    auto reach = [&](uint32_t bound) {
        if constexpr (BIAS) {
            // more than topk are not less than it by more than the error
            const float v = value(bound);
            if (bound > kNone) bound = number(v - 2.0f * error(v));
        }
        bound = more(bound, kNone + 1u);
        mine = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) mine |= key[c][d] >= bound ? 1u << (4 * c + d) : 0u;
        count = __popc(mine);
        behind = lanes_prefix<LPT>(count);
        n = (int)over_lanes32<LPT>((uint32_t)behind, more);
    };
    const bool lanes = LPT <= 16 && p.topk < LPT;
    if (lanes) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) m = more(m, key[c][d]);
        const int ahead = lanes_ahead<LPT>(m);
        // the smallest of the first topk + 1 (equal maxima count none of each other)
        reach(~over_lanes32<LPT>(~(ahead <= p.topk ? m : ~0u), more));
    }
    if (!lanes || __ballot(n > kRouteList)) {
        uint32_t m = 0;
        for (int r = 0; r <= p.topk; ++r) {
            uint32_t far = 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d) far = more(far, key[c][d] - m);
            const uint32_t next = over_lanes32<LPT>(far, more) + m;
            // none is left: every number is at or above m, or m was none
            m = r > 0 && (m <= kNone || next >= m) ? 0u : next;
        }
        reach(m);
    }

    // ---- the list of those that reach it, lane by lane ----
    for (int r = i; r < p.topk; r += LPT) {
        out[r] = 0xFFFFu;
        w[r] = 0.0f;
    }
    if (!__ballot(n > kRouteList)) {
        int at = behind - count;
        while (__ballot(mine != 0u)) {
            if (mine) {
                const int v = __ffs((int)mine) - 1;
                mine &= mine - 1u;
                es[at++] = (uint16_t)(4 * (i + LPT * (v / 4)) + v % 4);
            }
        }
        const int full = (n + 15) & ~15;                  // zeros are behind every entry
        for (int k = n + i; k < full; k += LPT) list[k] = 0;
        wave_order();
        for (int k = i; k < n; k += LPT) {
            const int e = es[k];
            const float b = BIAS ? p.bias[e] : 0.0f;
            const float v = cs[e], s = score(v);
            ss[k] = s;
            list[k] = (uint64_t)number(BIAS ? clean(s + b) : v + 0.0f) << 32 | (uint32_t)~e;
        }
        wave_order();
        for (int k = i; k < n; k += LPT) {
            const uint64_t own = list[k];
            const float s = ss[k];
            int place = 0;
            for (int h = 0; h < full; h += 16) {
                typedef uint64_t v2l __attribute__((ext_vector_type(2)));
                v2l u[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] = *reinterpret_cast<const v2l *>(list + h + 2 * q);
#pragma unroll
                for (int q = 0; q < 8; ++q) place += (u[q][0] > own ? 1 : 0) + (u[q][1] > own ? 1 : 0);
            }
            if (place < p.topk) {
                out[place] = (uint16_t)~(uint32_t)own;
                w[place] = s;
            }
        }
    } else {
        // ---- by (number, lower expert first), one a round ----
        if constexpr (BIAS) exact(kEvery);
        keys(doubt);
        for (int r = 0; r < p.topk; ++r) {
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d) m = more(m, key[c][d]);
            m = over_lanes32<LPT>(m, more);
            uint32_t won = ~0u;
#pragma unroll
            for (int c = C - 1; c >= 0; --c)
#pragma unroll
                for (int d = 3; d >= 0; --d)
                    won = key[c][d] == m ? (uint32_t)(4 * (i + LPT * c) + d) : won;
            won = ~over_lanes32<LPT>(~won, more);
            if (i == 0 && m > kNone) out[r] = (uint16_t)won;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (won == (uint32_t)(4 * (i + LPT * c) + d)) key[c][d] = 0u;
        }
        wave_order();
        for (int r = i; r < p.topk; r += LPT) {
            const int e = out[r];
            if (e != 0xFFFF) w[r] = score(logit(e));
        }
    }
    wave_order();

    // ---- ids and weights: lane r of the token writes choice r (and r + LPT, ..) ----
    // (their sum over the bits of r, in the order of the sums above)
    constexpr int R = (kRouteMaxTopk + LPT - 1) / LPT;
    int id[R];
    float v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int r = i + LPT * q;
        id[q] = r < p.topk ? out[r] : 0xFFFF;
        v[q] = r < p.topk ? w[r] : 0.0f;
    }
    float sum = 1.0f;
    if (p.renorm) sum = lanes_sum<LPT>(chunk_sum(v));
    if (live)
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int r = i + LPT * q;
            if (r >= p.topk) break;
            p.ids[t * p.topk + r] = id[q] != 0xFFFF ? id[q] : -1;
            p.weights[t * p.topk + r] = sum > 0.0f ? p.scale * (v[q] / sum) : 0.0f;
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
                     reinterpret_cast<uintptr_t>(a.logits) % (4 * size) == 0 &&
                     reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
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
