// mx_block.hip -- what lies between two blocks of a layer, in one pass over the rows:
//
//   p[m][k] = x[m][k] * rsqrt(mean_k x[m][k]^2 + eps) * (offset + post[k])
//   s[m][k] = T(alpha * residual[m][k] + gate[g][k] * p[m][k])      T bf16 or fp32
//   y[m][k] = bf16(s[m][k] * rsqrt(mean_k s[m][k]^2 + eps) * (offset + weight[k]))
//   (q, c)  = the MXFP8 bytes and codes of y (rule as in mx_quant.hip)
// Everything is fp32 between the inputs and the roundings written above: s is rounded
// before it is squared, as the rounded value is what the residual stream holds from
// then on, and y before it is quantized, so that the bytes are those of quantizing a
// stored y; p is not rounded (it never leaves the registers).
//
// Work split: a row is cut into segments of 512 values, eight a lane; WPR wavefronts
// share a row, wavefront w taking segments w, w + WPR, ...  Short rows take fewer
// wavefronts, and a workgroup of eight then holds 8 / WPR rows.  The row stays in
// registers through both sums.  The order of the sums is fixed by K: a lane's values
// in order, the 64 lanes by DPP and lane-swap steps, the row's wavefronts as a tree.
// T16 output: the rows of a 16-token tile go to workgroups of one XCD, whose L2 then
// merges their 16-byte pieces of each 128-byte line.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_lanes.h"

namespace mx {

constexpr int kBlockWaves = 8;             // wavefronts of a workgroup

template <int AUX = 0>
__device__ inline void put16(__amdgpu_buffer_rsrc_t r, v4u v, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, AUX);
}

// the sums of a row's WPR wavefronts, as a tree
template <int WPR>
__device__ inline float row_sum(float v, float *red, int wave) {
    if constexpr (WPR == 1) return v;
    if (threadIdx.x % 64 == 0) red[wave] = v;
    __syncthreads();
    const float *r = red + wave / WPR * WPR;
    float t[WPR];
#pragma unroll
    for (int c = 0; c < WPR; ++c) t[c] = r[c];
#pragma unroll
    for (int n = WPR / 2; n >= 1; n /= 2)
#pragma unroll
        for (int c = 0; c < n; ++c) t[c] += t[c + n];
    return t[0];
}

__device__ inline float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ inline float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// at most NS segments a wavefront; ACT as in mx_act; F32: the residual stream's type
template <int NS, int WPR, int ACT, int RULE, bool F32>
__global__ void __launch_bounds__(64 * kBlockWaves) block_norm_kernel(BlockNormArgs p) {
    constexpr int ROWS = kBlockWaves / WPR;               // rows of a workgroup
    __shared__ float red[2][kBlockWaves];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int w = wave % WPR;
    int64_t m = (int64_t)blockIdx.x * ROWS + wave / WPR;
    if (ACT == ACT_MXFP8_T16) {
        // the workgroups of a tile, W of them, have one number modulo 8
        constexpr int W = 16 / ROWS;
        const int64_t b = blockIdx.x;
        m = 16 * (b / (8 * W) * 8 + b % 8) + b / 8 % W * ROWS + wave / WPR;
        if (m / 16 >= (p.M + 15) / 16) return;            // the whole workgroup
    }
    const int K = (int)p.K;
    const bool live = m < p.M;                            // T16: rows past M pad the last tile
    const uint32_t rowb = live ? (uint32_t)K * 2u : 0u;
    const int64_t mr = live ? m : 0;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + mr * p.ldx, rowb);
    constexpr int SIZE = F32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(
        p.res ? static_cast<const uint8_t *>(p.res) + mr * p.ldr * SIZE : nullptr,
        p.res ? rowb / 2 * SIZE : 0u);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(
        p.sum ? static_cast<uint8_t *>(p.sum) + mr * p.lds * SIZE : nullptr,
        p.sum ? rowb / 2 * SIZE : 0u);
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(p.post, p.post ? (uint32_t)K * 2u : 0u);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.weight, p.weight ? (uint32_t)K * 2u : 0u);
    // a gate's number outside [0, gates): the block adds nothing
    int64_t gid = 0;
    if (p.gate && p.gate_ids && live) gid = p.gate_ids[m];
    const bool gated_out = p.gate && (gid < 0 || gid >= p.gates);
    const __amdgpu_buffer_rsrc_t gr = make_rsrc(
        p.gate ? p.gate + (gated_out ? 0 : gid) * p.ldg : nullptr, p.gate ? (uint32_t)K * 2u : 0u);

    v4u x[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        x[i] = load16<kNT>(xr, (uint32_t)(1024 * (w + WPR * i) + 16 * lane));
    v4u res[NS][F32 ? 2 : 1];
    if (p.res) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int h = 0; h < (F32 ? 2 : 1); ++h)
                res[i][h] = load16<kNT>(
                    rr, (uint32_t)((1024 * (w + WPR * i) + 16 * lane) * (SIZE / 2) + 16 * h));
    }

    float rstd = 1.0f;
    if (p.post) {
        float acc = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float lo = lo_f(x[i][d]), hi = hi_f(x[i][d]);
                acc = __builtin_fmaf(lo, lo, acc);
                acc = __builtin_fmaf(hi, hi, acc);
            }
        const float ss = row_sum<WPR>(lanes_sum<64>(acc), red[0], wave);
        rstd = 1.0f / __builtin_sqrtf(ss / (float)K + p.eps);
    }

    // the new residual stream, rounded to its type: bf16 pairs in x, or fp32 values
    float f[F32 ? NS : 1][F32 ? 8 : 1];
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const uint32_t off = (uint32_t)(1024 * (w + WPR * i) + 16 * lane);
        v4u pw = {0u, 0u, 0u, 0u}, gw = {0u, 0u, 0u, 0u};
        if (p.post) pw = load16(pr, off);
        if (p.gate) gw = load16(gr, off);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a = k % 2 ? hi_f(x[i][k / 2]) : lo_f(x[i][k / 2]);
            if (p.post) a = a * rstd * (p.offset + (k % 2 ? hi_f(pw[k / 2]) : lo_f(pw[k / 2])));
            if (p.gate) {
                a *= k % 2 ? hi_f(gw[k / 2]) : lo_f(gw[k / 2]);
                if (gated_out) a = 0.0f;
            }
            if (p.res) {
                const float r = F32 ? __uint_as_float(res[i][k / 4 % (F32 ? 2 : 1)][k % 4])
                                    : (k % 2 ? hi_f(res[i][0][k / 2]) : lo_f(res[i][0][k / 2]));
                a = __builtin_fmaf(p.alpha, r, a);
            }
            v[k] = a;
        }
        if constexpr (F32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[i][k] = v[k];
                acc = __builtin_fmaf(v[k], v[k], acc);
            }
            if (p.sum)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    put16<kNT>(sr, v4u{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                       __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])},
                               2 * off + 16u * h);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t u = bf16_bits(v[2 * d]) | bf16_bits(v[2 * d + 1]) << 16;
                x[i][d] = u;
                acc = __builtin_fmaf(lo_f(u), lo_f(u), acc);
                acc = __builtin_fmaf(hi_f(u), hi_f(u), acc);
            }
            if (p.sum) put16<kNT>(sr, x[i], off);
        }
    }
    if (!p.weight) return;                                // uniform: no second norm
    const float ss = row_sum<WPR>(lanes_sum<64>(acc), red[1], wave);
    const float scale = 1.0f / __builtin_sqrtf(ss / (float)K + p.eps);

    const __amdgpu_buffer_rsrc_t yr = make_rsrc(
        p.y ? p.y + mr * p.ldy : nullptr, p.y ? rowb : 0u);
    const int S = (K + 127) / 128, Q = (S + 3) / 4;
    const int r = (int)(m % 16);
    uint8_t *qbase = nullptr, *cbase = nullptr;
    uint32_t qbytes = 0;
    if (ACT == ACT_MXFP8) {
        qbase = p.xq + mr * p.ldq;
        qbytes = live ? (uint32_t)K : 0u;
        cbase = p.xcodes + mr * p.ldc;
    } else if (ACT == ACT_MXFP8_T16) {
        qbase = p.xq + m / 16 * S * 2048;
        qbytes = (uint32_t)S * 2048u;
        cbase = p.xcodes + m / 16 * Q * 256;
    }
    const __amdgpu_buffer_rsrc_t qr = make_rsrc(qbase, qbytes);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = w + WPR * i;                                // segment
        const int k0 = 512 * c + 8 * lane;
        const v4u wt = load16(wr, (uint32_t)(2 * k0));
        v4u o;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float a = F32 ? f[F32 ? i : 0][F32 ? 2 * d : 0] : lo_f(x[i][d]);
            const float b = F32 ? f[F32 ? i : 0][F32 ? 2 * d + 1 : 0] : hi_f(x[i][d]);
            const float lo = a * scale * (p.offset + lo_f(wt[d]));
            const float hi = b * scale * (p.offset + hi_f(wt[d]));
            // padding rows, and values past K: +0
            o[d] = live && k0 < K ? bf16_bits(lo) | bf16_bits(hi) << 16 : 0u;
        }
        if (p.y) put16(yr, o, (uint32_t)(2 * k0));
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
            if (lane % 4 == 0 && c < Q)
                cbase[c * 256 + 4 * (16 * (b % 4) + r) + b / 4] =
                    (uint8_t)(live && k0 < K ? code : 127u);
        }
        __builtin_amdgcn_raw_buffer_store_b64(q, qr, (int)off, 0, 0);
    }
}

template <int NS, int WPR, int ACT, bool F32>
static hipError_t launch_rule(const BlockNormArgs &a, int rule, hipStream_t st) {
    constexpr int ROWS = kBlockWaves / WPR;
    int64_t groups = (a.M + ROWS - 1) / ROWS;
    if (ACT == ACT_MXFP8_T16) groups = ((a.M + 15) / 16 + 7) / 8 * 8 * (16 / ROWS);
    const dim3 grid((unsigned)groups), block(64 * kBlockWaves);
    // (a bf16 output does not depend on the rule)
    if (ACT == ACT_BF16 || rule == RULE_OCP)
        hipLaunchKernelGGL((block_norm_kernel<NS, WPR, ACT, RULE_OCP, F32>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((block_norm_kernel<NS, WPR, ACT, RULE_CEIL448, F32>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <int NS, int WPR>
static hipError_t launch_act(const BlockNormArgs &a, int type, int act, int rule, hipStream_t st) {
    if (type == FLOAT_F32) {
        if (act == ACT_BF16) return launch_rule<NS, WPR, ACT_BF16, true>(a, rule, st);
        if (act == ACT_MXFP8) return launch_rule<NS, WPR, ACT_MXFP8, true>(a, rule, st);
        return launch_rule<NS, WPR, ACT_MXFP8_T16, true>(a, rule, st);
    }
    if (act == ACT_BF16) return launch_rule<NS, WPR, ACT_BF16, false>(a, rule, st);
    if (act == ACT_MXFP8) return launch_rule<NS, WPR, ACT_MXFP8, false>(a, rule, st);
    return launch_rule<NS, WPR, ACT_MXFP8_T16, false>(a, rule, st);
}

hipError_t launch_block_norm(const BlockNormArgs &a, int type, int act, int rule, hipStream_t st) {
    const int64_t segs = (a.K + 511) / 512;
    if (segs <= 1) return launch_act<1, 1>(a, type, act, rule, st);
    if (segs <= 2) return launch_act<1, 2>(a, type, act, rule, st);
    if (segs <= 4) return launch_act<1, 4>(a, type, act, rule, st);
    if (segs <= 8) return launch_act<1, 8>(a, type, act, rule, st);
    if (segs <= 16) return launch_act<2, 8>(a, type, act, rule, st);
    if (segs <= 32) return launch_act<4, 8>(a, type, act, rule, st);
    if (segs <= 64) return launch_act<8, 8>(a, type, act, rule, st);
    return launch_act<16, 8>(a, type, act, rule, st);
}

}  // namespace mx
