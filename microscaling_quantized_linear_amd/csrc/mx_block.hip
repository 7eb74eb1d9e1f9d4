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
//
// Bound: the bytes.  4096 rows of 7168 with an fp32 residual stream, 383 MB: 72 us,
// 5.3 TB/s (a large copy: 4.75); a bf16 stream, 265 MB: 49 us, 5.4 TB/s.  One row or eight:
// the launch and three trips to memory, 4.7 us.  What was measured for it and left out, at
// the first of these sizes: the norms' vectors loaded ahead with the row 77 us (more
// registers, fewer rows in flight); two workgroups a compute unit that go over the rows
// with the next one's loads in flight 85 us.  Rows of more than 32768 values keep 16
// segments a wavefront: with an fp32 stream that spills 88 to 96 bytes a lane (512 rows of
// 65536, 436 MB 109 us, 4.0 TB/s; 32768 47 us, 4.6; bf16 61 and 31).
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_lanes.h"

namespace mx {

constexpr int kBlockWaves = 8;             // wavefronts of a workgroup
// x and the residual together, up to which they are loaded through the caches (the figure
// lies between two that were measured, 55.7 and 58.7 MB): a chain of such calls stays in
// the 256 MB of Infinity Cache (5001 rows of 1568, 31 and 47 MB:
// 13.0 against 15.0 us, fp32 stream 18.7 against 21.9; 3400 of 4096, 56 MB: 20.4 against
// 23.1).  Larger ones go past them (4096 rows of 7168, 117 MB: 49.2 against 54.4 us; 2048
// rows, 59 MB: 28.7 against 29.7).
constexpr int64_t kCachedBytes = 56000000;

template <int AUX = 0>
__device__ inline void put16(__amdgpu_buffer_rsrc_t r, v4u v, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, AUX);
}

// A row's sum.  Its segments' numbers modulo CL make CL classes; wavefront w of the
// row's WPR holds CL / WPR of them, v[i] being its lanes' sums of class w + WPR i.
// The lanes are added first, then the classes as a tree: the same order for every WPR.
template <int WPR, int CL>
__device__ inline float row_sum(const float (&v)[CL / WPR], float *red, int wave) {
    constexpr int PER = CL / WPR;
    float t[PER > WPR ? PER : WPR];
#pragma unroll
    for (int i = 0; i < PER; ++i) t[i] = lanes_sum<64>(v[i]);
#pragma unroll
    for (int n = PER / 2; n >= 1; n /= 2)
#pragma unroll
        for (int c = 0; c < n; ++c) t[c] += t[c + n];
    if constexpr (WPR == 1) return t[0];
    if (threadIdx.x % 64 == 0) red[wave] = t[0];
    __syncthreads();
    const float *r = red + wave / WPR * WPR;
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

// at most NS segments a wavefront, in CL classes a row; ACT as in mx_act; F32: the
// residual stream's type; NT: x and the residual go past the caches
template <int NS, int WPR, int CL, int ACT, bool F32, bool NT>
__global__ void __launch_bounds__(64 * kBlockWaves) block_norm_kernel(BlockNormArgs p) {
    constexpr int ROWS = kBlockWaves / WPR;               // rows of a workgroup
    constexpr int PER = CL / WPR;
    static_assert(NS % PER == 0, "whole classes");
    constexpr int SIZE = F32 ? 4 : 2, RN = F32 ? 2 : 1, AUX = NT ? kNT : 0;
    __shared__ float red[2][kBlockWaves];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int w = wave % WPR;
    const int K = (int)p.K, S = (K + 127) / 128, Q = (S + 3) / 4;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.weight, p.weight ? (uint32_t)K * 2u : 0u);
    auto seg = [&](int i) -> uint32_t { return (uint32_t)(1024 * (w + WPR * i) + 16 * lane); };

    int64_t m = (int64_t)blockIdx.x * ROWS + wave / WPR;
    if (ACT == ACT_MXFP8_T16) {
        // the groups of a tile, W of them, have one number modulo 8
        constexpr int W = 16 / ROWS;
        const int64_t b = blockIdx.x;
        m = 16 * (b / (8 * W) * 8 + b % 8) + b / 8 % W * ROWS + wave / WPR;
    }
    const bool live = m < p.M;                            // T16: rows past M pad the last tile
    const uint32_t rowb = live ? (uint32_t)K * 2u : 0u;
    const int64_t mr = live ? m : 0;
    // a gate's number outside [0, gates): the block adds nothing.  x reads as zeros, and
    // neither a gate nor the post weight is there (their infinities would make NaN of it)
    int64_t gid = 0;
    if (p.gate && p.gate_ids && live) gid = p.gate_ids[m];
    const bool out = p.gate && (gid < 0 || gid >= p.gates);
    // What is not there costs no branch: an empty resource reads zeros, the vectors'
    // offset is then 1.
    const bool post = p.post && !out, gated = p.gate && !out;
    const float poff = post ? p.offset : 1.0f, goff = gated ? 0.0f : 1.0f;
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(p.post, post ? (uint32_t)K * 2u : 0u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + mr * p.ldx, out ? 0u : rowb);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(
        p.res ? static_cast<const uint8_t *>(p.res) + mr * p.ldr * SIZE : nullptr,
        p.res ? rowb / 2 * SIZE : 0u);
    const __amdgpu_buffer_rsrc_t gr = make_rsrc(
        p.gate ? p.gate + (out ? 0 : gid) * p.ldg : nullptr, gated ? (uint32_t)K * 2u : 0u);
    v4u x[NS], res[NS][RN], gate[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] = load16<AUX>(xr, seg(i));
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int h = 0; h < RN; ++h)
            res[i][h] = load16<AUX>(rr, seg(i) * (SIZE / 2) + 16u * h);
#pragma unroll
    for (int i = 0; i < NS; ++i) gate[i] = load16(gr, seg(i));

    float rstd = 1.0f;
    if (p.post) {
        float acc[PER] = {};
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float lo = lo_f(x[i][d]), hi = hi_f(x[i][d]);
                acc[i % PER] = __builtin_fmaf(lo, lo, acc[i % PER]);
                acc[i % PER] = __builtin_fmaf(hi, hi, acc[i % PER]);
            }
        const float ss = row_sum<WPR, CL>(acc, red[0], wave);
        rstd = out ? 0.0f : 1.0f / __builtin_sqrtf(ss / (float)K + p.eps);
    }

    // the new residual stream, rounded to its type: bf16 pairs in x, or fp32 values
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(
        p.sum ? static_cast<uint8_t *>(p.sum) + mr * p.lds * SIZE : nullptr,
        p.sum ? rowb / 2 * SIZE : 0u);
    float f[F32 ? NS : 1][F32 ? 8 : 1];
    float acc[PER] = {};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const v4u pw = load16(pr, seg(i));
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            auto half = [&](const v4u &u) { return k % 2 ? hi_f(u[k / 2]) : lo_f(u[k / 2]); };
            const float r = F32 ? __uint_as_float(res[i][F32 ? k / 4 : 0][k % 4])
                                : half(res[i][0]);
            const float n = half(x[i]) * rstd * (poff + half(pw)) * (goff + half(gate[i]));
            v[k] = __builtin_fmaf(p.alpha, r, n);
        }
        if constexpr (F32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[i][k] = v[k];
                acc[i % PER] = __builtin_fmaf(v[k], v[k], acc[i % PER]);
            }
            if (p.sum)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    put16<kNT>(sr,
                               v4u{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                   __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])},
                               2 * seg(i) + 16u * h);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t u = bf16_bits(v[2 * d]) | bf16_bits(v[2 * d + 1]) << 16;
                x[i][d] = u;
                acc[i % PER] = __builtin_fmaf(lo_f(u), lo_f(u), acc[i % PER]);
                acc[i % PER] = __builtin_fmaf(hi_f(u), hi_f(u), acc[i % PER]);
            }
            if (p.sum) put16<kNT>(sr, x[i], seg(i));
        }
    }
    if (p.weight) {                                   // uniform: else no second norm
        const float ss = row_sum<WPR, CL>(acc, red[1], wave);
        const float scale = 1.0f / __builtin_sqrtf(ss / (float)K + p.eps);
        const __amdgpu_buffer_rsrc_t yr = make_rsrc(
            p.y ? p.y + mr * p.ldy : nullptr, p.y ? rowb : 0u);
        const int64_t mb = m / 16;
        const int r = (int)(m % 16);
        uint8_t *qbase = nullptr, *cbase = nullptr;
        uint32_t qbytes = 0;
        if (ACT == ACT_MXFP8) {
            qbase = p.xq + mr * p.ldq;
            qbytes = live ? (uint32_t)K : 0u;
            cbase = p.xcodes + mr * p.ldc;
        } else if (ACT == ACT_MXFP8_T16) {
            const bool tile = mb < (p.M + 15) / 16;
            qbase = p.xq + (tile ? mb * S * 2048 : 0);
            qbytes = tile ? (uint32_t)S * 2048u : 0u;
            cbase = tile ? p.xcodes + mb * Q * 256 : nullptr;
        }
        const __amdgpu_buffer_rsrc_t qr = make_rsrc(qbase, qbytes);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = w + WPR * i;                        // segment
            const int k0 = 512 * c + 8 * lane;
            const v4u wt = load16(wr, seg(i));
            v4u o;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float lo = F32 ? f[F32 ? i : 0][F32 ? 2 * d : 0] : lo_f(x[i][d]);
                const float hi = F32 ? f[F32 ? i : 0][F32 ? 2 * d + 1 : 0] : hi_f(x[i][d]);
                o[d] = bf16_bits(lo * scale * (p.offset + lo_f(wt[d]))) |
                       bf16_bits(hi * scale * (p.offset + hi_f(wt[d]))) << 16;
                // the tile's padding rows, and values past K: +0 (elsewhere not stored)
                if (ACT == ACT_MXFP8_T16 && !(live && k0 < K)) o[d] = 0u;
            }
            if (p.y) put16(yr, o, (uint32_t)(2 * k0));
            if (ACT == ACT_BF16) continue;
            uint32_t code;
            v2u q;
            if (p.rule == RULE_OCP) q = quant_eighth<RULE_OCP>(o, code);   // uniform
            else q = quant_eighth<RULE_CEIL448>(o, code);
            uint32_t off;
            if (ACT == ACT_MXFP8) {
                off = (uint32_t)k0;
                if (lane % 4 == 0 && live && k0 < K) cbase[k0 / 32] = (uint8_t)code;
            } else {
                // step s, half h, lane group j, byte c8 of the 16-byte piece
                off = (uint32_t)((k0 / 64) * 1024 + (k0 % 64 / 16) * 256 + 16 * r + k0 % 16);
                // block 16 c + b of the row: lane group b % 4, byte b / 4 of quad c
                const int blk = lane / 4;
                if (lane % 4 == 0 && cbase && c < Q)
                    cbase[c * 256 + 4 * (16 * (blk % 4) + r) + blk / 4] =
                        (uint8_t)(live && k0 < K ? code : 127u);
            }
            __builtin_amdgcn_raw_buffer_store_b64(q, qr, (int)off, 0, 0);
        }
    }
}

template <int NS, int WPR, int CL, int ACT, bool F32>
static hipError_t launch_nt(const BlockNormArgs &a, hipStream_t st) {
    constexpr int ROWS = kBlockWaves / WPR;
    int64_t groups = (a.M + ROWS - 1) / ROWS;
    if (ACT == ACT_MXFP8_T16) groups = ((a.M + 15) / 16 + 7) / 8 * 8 * (16 / ROWS);
    const dim3 grid((unsigned)groups), block(64 * kBlockWaves);
    if (a.M * a.K * (F32 ? 6 : 4) > kCachedBytes)
        hipLaunchKernelGGL((block_norm_kernel<NS, WPR, CL, ACT, F32, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((block_norm_kernel<NS, WPR, CL, ACT, F32, false>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <int NS, int WPR, int CL>
static hipError_t launch_act(const BlockNormArgs &a, int type, int act, hipStream_t st) {
    if (type == FLOAT_F32) {
        if (act == ACT_BF16) return launch_nt<NS, WPR, CL, ACT_BF16, true>(a, st);
        if (act == ACT_MXFP8) return launch_nt<NS, WPR, CL, ACT_MXFP8, true>(a, st);
        return launch_nt<NS, WPR, CL, ACT_MXFP8_T16, true>(a, st);
    }
    if (act == ACT_BF16) return launch_nt<NS, WPR, CL, ACT_BF16, false>(a, st);
    if (act == ACT_MXFP8) return launch_nt<NS, WPR, CL, ACT_MXFP8, false>(a, st);
    return launch_nt<NS, WPR, CL, ACT_MXFP8_T16, false>(a, st);
}

hipError_t launch_block_norm(const BlockNormArgs &a, int type, int act, hipStream_t st) {
    const int64_t segs = (a.K + 511) / 512;
    if (segs <= 1) return launch_act<1, 1, 1>(a, type, act, st);
    if (segs <= 2) return launch_act<1, 2, 2>(a, type, act, st);
    if (segs <= 4) return launch_act<1, 4, 4>(a, type, act, st);
    if (segs <= 8) return launch_act<1, 8, 8>(a, type, act, st);
    if (segs <= 16) return launch_act<2, 8, 8>(a, type, act, st);
    if (segs <= 32) return launch_act<4, 8, 8>(a, type, act, st);
    if (segs <= 64) return launch_act<8, 8, 8>(a, type, act, st);
    return launch_act<16, 8, 8>(a, type, act, st);
}

}  // namespace mx
