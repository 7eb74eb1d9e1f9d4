// mx_norm.hip -- residual addition, root-mean-square norm and the norm's
// output as an MXFP8 activation, in one pass over the rows.
//
//   s[m][k] = bf16(x[m][k] + residual[m][k])
//   y[m][k] = bf16(s[m][k] * rsqrt(mean_k s[m][k]^2 + eps) * weight[k])
//   (q, c)  = the MXFP8 bytes and codes of y (rule as in mx_quant.hip)
// The sum and its norm are formed in fp32.  s is rounded to bf16 before it is
// squared because the rounded value is what the residual stream holds from
// then on, and y before it is quantized because the bytes then equal those of
// quantizing a stored bf16 y: a caller may switch between the two forms
// without a change in its results.
//
// Work split: a row is cut into segments of 512 values, eight a lane (one
// 16-byte load of x and one of the residual).  Eight wavefronts share a row,
// wavefront w taking segments w, w + 8, ...; the row stays in registers
// between the sum of squares and the output, so x and the residual are read
// once.  A quad of lanes holds one 32-value block, so the block maximum is two
// DPP steps, and a segment is exactly one quad of 128-K steps of the T16
// layout: a lane pair writes 16 contiguous bytes of it.
// x, the residual and the stored sum go past the caches (the sum is next read a
// layer later): M = 4096, K = 7168 with every output, 265 MB, 48.5 -> 42.5 us,
// 6.2 TB/s (T16 output without y, 207 MB: 55.5 us, its stores are 16-byte pieces of
// lines that eight XCDs share); y and the bytes, which the next product reads, do not.
// The order of the sum of squares is fixed by K: a lane's values, the eight
// wavefronts as a tree, then the 64 lanes.  A row's result is therefore the same
// in any call.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

// loads and stores past the resource's end read zeros / are dropped, so a
// ragged last segment takes no branch
template <int AUX = 0>
__device__ inline void store16(__amdgpu_buffer_rsrc_t r, v4u v, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, AUX);
}

constexpr int kRowWaves = 8;               // wavefronts, and one row a workgroup

// at most NS segments a wavefront; ACT as in mx_act
template <int NS, int ACT, int RULE>
__global__ void __launch_bounds__(64 * kRowWaves) add_rms_norm_kernel(NormArgs p) {
    const int lane = threadIdx.x % 64;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t m = blockIdx.x;
    const int K = (int)p.K;
    const bool live = m < p.M;                            // T16: rows past M pad the last tile
    const uint32_t rowb = live ? (uint32_t)K * 2u : 0u;
    const int64_t mr = live ? m : 0;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + mr * p.ldx, rowb);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(
        p.res ? p.res + mr * p.ldr : p.x, p.res ? rowb : 0u);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(
        p.sum ? p.sum + mr * p.lds : nullptr, p.sum ? rowb : 0u);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.weight, (uint32_t)K * 2u);

    v4u v[NS], wt[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        v[i] = load16<kNT>(xr, (uint32_t)(1024 * (w + kRowWaves * i) + 16 * lane));
    v4u res[NS];
    if (p.res) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            res[i] = load16<kNT>(rr, (uint32_t)(1024 * (w + kRowWaves * i) + 16 * lane));
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
        wt[i] = load16(wr, (uint32_t)(1024 * (w + kRowWaves * i) + 16 * lane));

    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t u = v[i][d];
            if (p.res) {
                const float lo = __uint_as_float(u << 16) + __uint_as_float(res[i][d] << 16);
                const float hi = __uint_as_float(u & 0xFFFF0000u) +
                                 __uint_as_float(res[i][d] & 0xFFFF0000u);
                u = bf16_bits(lo) | bf16_bits(hi) << 16;
                v[i][d] = u;
            }
            const float lo = __uint_as_float(u << 16), hi = __uint_as_float(u & 0xFFFF0000u);
            acc = __builtin_fmaf(lo, lo, acc);
            acc = __builtin_fmaf(hi, hi, acc);
        }
        if (p.sum) store16<kNT>(sr, v[i], (uint32_t)(1024 * (w + kRowWaves * i) + 16 * lane));
    }
    __shared__ float red[kRowWaves][64];
    red[w][lane] = acc;
    __syncthreads();
    float t[kRowWaves];
#pragma unroll
    for (int c = 0; c < kRowWaves; ++c) t[c] = red[c][lane];
    float ss = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o);
    const float scale = 1.0f / __builtin_sqrtf(ss / (float)K + p.eps);

    const __amdgpu_buffer_rsrc_t yr = make_rsrc(
        p.y ? p.y + mr * p.ldy : nullptr, p.y ? rowb : 0u);
    // quantized output: the row's bytes (row-major) or its token tile (T16)
    const int S = (K + 127) / 128, Q = (S + 3) / 4;
    const int64_t mb = m / 16;
    const int r = (int)(m % 16);
    uint8_t *qbase = nullptr, *cbase = nullptr;
    uint32_t qbytes = 0;
    if (ACT == ACT_MXFP8) {
        qbase = p.xq + m * p.ldq;
        qbytes = live ? (uint32_t)K : 0u;
        cbase = p.xcodes + m * p.ldc;
    } else if (ACT == ACT_MXFP8_T16) {
        const bool tile = mb < (p.M + 15) / 16;
        qbase = p.xq + (tile ? mb * S * 2048 : 0);
        qbytes = tile ? (uint32_t)S * 2048u : 0u;
        cbase = tile ? p.xcodes + mb * Q * 256 : nullptr;
    }
    const __amdgpu_buffer_rsrc_t qr = make_rsrc(qbase, qbytes);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = w + kRowWaves * i;                          // segment
        const int k0 = 512 * c + 8 * lane;
        v4u o;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float lo = __uint_as_float(v[i][d] << 16) * scale *
                             __uint_as_float(wt[i][d] << 16);
            const float hi = __uint_as_float(v[i][d] & 0xFFFF0000u) * scale *
                             __uint_as_float(wt[i][d] & 0xFFFF0000u);
            // padding rows, and values past K (which the scale of a row that is not
            // finite would turn into NaN): +0
            o[d] = live && k0 < K ? bf16_bits(lo) | bf16_bits(hi) << 16 : 0u;
        }
        if (p.y) store16(yr, o, (uint32_t)(2 * k0));
        if (ACT == ACT_BF16) continue;
        uint32_t code;
        const v2u q = quant_eighth<RULE>(o, code);
        uint32_t off;
        if (ACT == ACT_MXFP8) {
            off = (uint32_t)k0;
            if (lane % 4 == 0 && live && k0 < K) cbase[k0 / 32] = (uint8_t)code;
        } else {
            // step s, half h, lane group j, byte c8 of the 16-byte piece
            off = (uint32_t)((k0 / 64) * 1024 + (k0 % 64 / 16) * 256 + 16 * r + k0 % 16);
            // block 16 c + b of the row: lane group b % 4, byte b / 4 of quad c
            const int b = lane / 4;
            if (lane % 4 == 0 && cbase && c < Q)
                cbase[c * 256 + 4 * (16 * (b % 4) + r) + b / 4] =
                    (uint8_t)(live && k0 < K ? code : 127u);
        }
        __builtin_amdgcn_raw_buffer_store_b64(q, qr, (int)off, 0, 0);
    }
}

template <int NS, int ACT>
static hipError_t launch_rule(const NormArgs &a, int64_t rows, int rule, hipStream_t st) {
    const dim3 grid((unsigned)rows), block(64 * kRowWaves);
    if (rule == RULE_OCP)
        hipLaunchKernelGGL((add_rms_norm_kernel<NS, ACT, RULE_OCP>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((add_rms_norm_kernel<NS, ACT, RULE_CEIL448>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <int NS>
static hipError_t launch_act(const NormArgs &a, int64_t rows, int act, int rule, hipStream_t st) {
    // (a bf16 output does not depend on the rule)
    if (act == ACT_BF16) return launch_rule<NS, ACT_BF16>(a, rows, RULE_OCP, st);
    if (act == ACT_MXFP8) return launch_rule<NS, ACT_MXFP8>(a, rows, rule, st);
    return launch_rule<NS, ACT_MXFP8_T16>(a, rows, rule, st);
}

hipError_t launch_add_rms_norm(const NormArgs &a, int act, int rule, hipStream_t st) {
    const int64_t segs = (a.K + 511) / 512;
    const int64_t rows = act == ACT_MXFP8_T16 ? (a.M + 15) / 16 * 16 : a.M;
    if (segs <= 8) return launch_act<1>(a, rows, act, rule, st);
    if (segs <= 16) return launch_act<2>(a, rows, act, rule, st);
    if (segs <= 32) return launch_act<4>(a, rows, act, rule, st);
    if (segs <= 64) return launch_act<8>(a, rows, act, rule, st);
    return launch_act<16>(a, rows, act, rule, st);
}

}  // namespace mx
