// mx_grouped.hip -- products grouped by expert over ragged row ranges:
//
//   y[i][n] = sum_k a[i][k] dec(W[e][n][k]) 2^(code - 127)
//             for offsets[e] <= i < offsets[e + 1],  a MXFP8 in the T16 layout
//   (EPI)  h[i][n] = silu(y[i][2 n]) * y[i][2 n + 1], one rounding
// e4m3 and e2m1 weights both run on the scaled matrix cores against the e4m3
// activations (v_mfma_scale_f32_16x16x128_f8f6f4 takes a format for each
// operand), with the E8M0 codes as lane scales.  The instruction adds the products
// of eight neighbouring K values in fixed point, with a last place of 2^-13 of the
// binade of the largest, and these sums in fp32.  That is the linear's precision
// too, and taken here for its reason: a result moves by 3e-4 to 4e-4 of itself
// against sums in fp32, a fifth of the bf16 rounding that follows (distance from
// the exact result 1.7e-3 with either), and the bf16 instruction, whose products
// keep 2^-24, has half the rate and needs both operands decoded.
//
// Expert ranges start anywhere: a lane addresses its own token row in the T16
// layout (tile row / 16, slot row % 16), so no range is padded and no row is
// computed twice.  Offsets are read on the device; the host knows their bound
// M only.  Rows of y behind offsets[E] are not written.
//
// Weight-streaming form (this kernel).  One workgroup owns NT 16-row weight
// tiles of one expert and runs over the expert's rows in batches of 16 MT; its
// four wavefronts split the 128-K steps into contiguous ranges and add their
// partial tiles in LDS in a fixed order.  Weights stream once from HBM per
// batch; activations come from L2.  An expert without rows costs one load of
// its offsets.  NT = 2 for e4m3 and 4 for e2m1 keep as many bytes in flight and
// enough workgroups (E 32, 4096 x 4096, 4 rows an expert: e4m3 82 us, with NT 1
// 93 and 4 98; e2m1 44 us, 6.1 TB/s, with NT 2 52 and 8 64; eight wavefronts 102
// and 59, two 82 and 47).  The weights go past the caches where a batch mostly
// takes all of an expert's rows (82 us, with caches 89); batches of 64 rows read
// them again, from the caches (E 16, 2048 x 7168, 48 rows: 82 -> 61 us).
#include "mx_device.h"
#include "mx_kernels.h"

#include <cstdlib>

namespace mx {

constexpr int kStreamWaves = 4;

// e2m1 (A) x e4m3 (B) with per-lane E8M0 scales in byte 0 of sa / sb; the
// e2m1 operand is the first four registers: K 32 j .. 32 j + 31 of lane group j
__device__ inline v4f mfma_fp4_fp8_scaled(v4u a, v8i b, v4f c, int sa, int sb) {
    const v8i a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b, c, 4, 0, 0, sa, 0, sb);
}

__device__ inline float silu(float g) { return g / (1.0f + __expf(-g)); }

template <int ELEM, int MT, int NT>
struct StreamStep {
    v4u w0[NT], w1[ELEM == E4M3 ? NT : 1], x0[MT], x1[MT];
    uint32_t cw[NT], cx[MT];
};

template <int ELEM, int LAYOUT, int MT, int NT>
__global__ void __launch_bounds__(64 * kStreamWaves) grouped_stream_kernel(GroupedArgs p) {
    constexpr int kAux = MT == 4 ? 0 : kNT;
    __shared__ v4f red[kStreamWaves][NT * MT][64];
    const int64_t e = blockIdx.y;
    // ranges that break the rules are cut to [0, M)
    int64_t o0 = p.offsets[e], o1 = p.offsets[e + 1];
    o0 = o0 < 0 ? 0 : o0;
    o1 = o1 > p.M ? p.M : o1;
    if (o0 >= o1) return;
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int S = (int)((p.K + 127) / 128), Q = (S + 3) / 4;
    const int64_t T = p.N / 16, t0 = (int64_t)blockIdx.x * NT;
    const int nt = (int)(T - t0 < NT ? T - t0 : NT);
    constexpr int CHUNK = ELEM == E4M3 ? 2048 : 1024;
    const int64_t TILEB = 16 * (ELEM == E4M3 ? p.K : p.K / 2);
    const uint32_t tailb = (uint32_t)(TILEB - (int64_t)(S - 1) * CHUNK);
    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(p.w + (e * T + t0) * TILEB, (uint32_t)(nt * TILEB));
    // ROW32: the tiles' code dwords; BLK32: one dword a block and 32 rows
    const __amdgpu_buffer_rsrc_t cr =
        LAYOUT == ROW32 ? make_rsrc(p.codes + (e * T + t0) * Q * 256, (uint32_t)(nt * Q * 256))
                        : make_rsrc(p.codes + e * (p.N / 32) * Q * 16,
                                    (uint32_t)((p.N / 32) * Q * 16));
    const int s0 = wave * S / kStreamWaves, s1 = (wave + 1) * S / kStreamWaves;

    for (int64_t row0 = o0; row0 < o1; row0 += 16 * MT) {
        // the batch's token tiles: at most MT + 1, the first that of row0
        const int64_t mb0 = row0 / 16, mtiles = (p.M + 15) / 16 - mb0;
        const uint32_t nmb = (uint32_t)(mtiles < MT + 1 ? mtiles : MT + 1);
        const __amdgpu_buffer_rsrc_t xr =
            make_rsrc(p.xq + mb0 * S * 2048, nmb * (uint32_t)S * 2048u);
        const __amdgpu_buffer_rsrc_t xcr =
            make_rsrc(p.xct + mb0 * Q * 256, nmb * (uint32_t)Q * 256u);
        uint32_t xo[MT], xco[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t row = row0 + 16 * i + r;
            const uint32_t mb = (uint32_t)(row / 16 - mb0), slot = (uint32_t)(row % 16);
            xo[i] = row < o1 ? mb * (uint32_t)S * 2048u + 256u * j + 16u * slot : kOOB;
            xco[i] = row < o1 ? mb * (uint32_t)Q * 256u + 64u * j + 4u * slot : kOOB;
        }
        auto load = [&](int s) {
            StreamStep<ELEM, MT, NT> st;
            const uint32_t past = s < s1 ? 0u : kOOB;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t o = 16u * lane;
                const uint32_t base = (uint32_t)(t * TILEB + (int64_t)s * CHUNK) & ~kOOB;
                const bool last = s == S - 1;
                st.w0[t] = load16<kAux>(wr, (base + o) | past | (last && o >= tailb ? kOOB : 0u));
                if (ELEM == E4M3)
                    st.w1[t] = load16<kAux>(
                        wr, (base + 1024u + o) | past | (last && o + 1024u >= tailb ? kOOB : 0u));
                st.cw[t] = load4(cr, (LAYOUT == ROW32
                                          ? (uint32_t)(t * Q + s / 4) * 256u + 4u * lane
                                          : (uint32_t)((t0 + t) / 2 * Q + s / 4) * 16u + 4u * j) |
                                         past);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t off = (xo[i] & ~kOOB) + (uint32_t)s * 2048u;
                const uint32_t bad = (xo[i] & kOOB) | past;
                st.x0[i] = load16(xr, off | bad);
                st.x1[i] = load16(xr, (off + 1024u) | bad);
                st.cx[i] = load4(xcr, ((xco[i] & ~kOOB) + (uint32_t)(s / 4) * 256u) | bad);
            }
            return st;
        };
        v4f acc[NT][MT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
        auto use = [&](const StreamStep<ELEM, MT, NT> &st, int s) {
            const int sh = 8 * (s % 4);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const v8i b = cat8(st.x0[i], st.x1[i]);
                const int sb = (int)(st.cx[i] >> sh);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int sa = (int)(st.cw[t] >> sh);
                    if (ELEM == E4M3)
                        acc[t][i] = mfma_fp8_scaled(cat8(st.w0[t], st.w1[t]), b, acc[t][i], sa, sb);
                    else
                        acc[t][i] = mfma_fp4_fp8_scaled(st.w0[t], b, acc[t][i], sa, sb);
                }
            }
        };
        // two steps a round, the next round's loads issued ahead of its products
        StreamStep<ELEM, MT, NT> a0 = load(s0), a1 = load(s0 + 1);
        for (int s = s0; s < s1; s += 2) {
            const StreamStep<ELEM, MT, NT> b0 = load(s + 2), b1 = load(s + 3);
            use(a0, s);
            use(a1, s + 1);
            a0 = b0;
            a1 = b1;
        }
        if (row0 != o0) __syncthreads();                  // the last batch's partials are used up
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) red[wave][t * MT + i][lane] = acc[t][i];
        __syncthreads();
        // element i of lane (jj, rr): weight row 4 jj + i, token rr
        for (int n = threadIdx.x; n < MT * 16 * NT * 4; n += 64 * kStreamWaves) {
            const int jj = n % 4, t = n / 4 % NT, rr = n / (4 * NT) % 16, i = n / (64 * NT);
            const int64_t row = row0 + 16 * i + rr;
            v4f s = red[0][t * MT + i][16 * jj + rr];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) s += red[w][t * MT + i][16 * jj + rr];
            if (row >= o1 || t >= nt) continue;
            const int64_t col = 16 * (t0 + t) + 4 * jj;
            if (p.epi) {
                *reinterpret_cast<uint32_t *>(p.y + row * p.ldy + col / 2) =
                    bf16_bits(silu(s[0]) * s[1]) | bf16_bits(silu(s[2]) * s[3]) << 16;
            } else {
                *reinterpret_cast<v2u *>(p.y + row * p.ldy + col) =
                    v2u{bf16_bits(s[0]) | bf16_bits(s[1]) << 16,
                        bf16_bits(s[2]) | bf16_bits(s[3]) << 16};
            }
        }
    }
}

template <int ELEM, int LAYOUT, int NT>
static hipError_t launch_stream(const GroupedArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)((a.N / 16 + NT - 1) / NT), (unsigned)a.E), block(64 * kStreamWaves);
    const int64_t rows = a.M / a.E;                       // an expert's rows, on average
    if (rows <= 6)
        hipLaunchKernelGGL((grouped_stream_kernel<ELEM, LAYOUT, 1, NT>), grid, block, 0, st, a);
    else if (rows <= 20)
        hipLaunchKernelGGL((grouped_stream_kernel<ELEM, LAYOUT, 2, NT>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((grouped_stream_kernel<ELEM, LAYOUT, 4, NT>), grid, block, 0, st, a);
    return hipGetLastError();
}

// Which form serves a call: 0 streams the weights, 1 and 2 are the tiled form
// with tiles of up to 128 and 256 rows.  The host knows the rows' number, not
// their split: the rule goes by the average (in the batch-invariant mode the
// streaming form serves every call, as K alone fixes its order).  Measured (us, streaming / 128 /
// 256; e4m3 unless named):
//   an expert's rows      4            8            16           128
//   E 32, 4096 x 4096     83/92/92     94/95/95     100/95/95    352/126/115
//   the same, e2m1        44/50/50     55/55/54     57/56/56     218/92/82
//   E 24, 4096 x 1568     29/31/31     37/31        41/32/32
//   E 64, 512 x 2048      14/17/17                  23/18/18     75/21/28
// With fewer weight panels (of 256 rows) than half the compute units the tiled
// form's time is that of one tile, whatever the rows, until its tiles fill the
// chip.  The streaming form's grows with the batches of 64 rows, and with the
// panels where these are more than about 28 (streaming / 128; the 256-row tiles
// are slower up to 256 rows):
//   panels, batches of 64 rows    1        2        3        4
//   K 4096, e4m3   16             9/23     16/24    22/24    29/24
//                  32             13/23    21/24    30/25    38/25
//                  48             19/23    33/25    47/25    61/26
//                  64             22/24    37/25    51/26    66/26
//                  96             30/25    53/26    74/28    96/30
//                  120            36/27    64/28    92/33    121/34
//   the same, e2m1 16             8/21     13/22    18/22    23/22
//                  48             13/22    24/23    33/24    42/24
//                  96             22/22    38/24    54/25    70/27
//   K 1024, e4m3   16             7/10     8/11     11/11    14/11
//                  48             8/10     14/11    21/12    27/12
//                  96             13/11    24/12    33/13    42/14
// They meet near 90 panel batches, and batches of at most 16 rows, whose
// products cost little, stream at any of these panels (96: 22/24, 120: 24/27).
// MX_GROUPED_FORM (1 to 3) overrides the rule (tuning sweeps only; read once).
static int grouped_form(const GroupedArgs &a) {
    static const int forced = [] {
        const char *s = std::getenv("MX_GROUPED_FORM");
        return s ? std::atoi(s) : 0;
    }();
    if (a.invariant || a.E > kGroupedMaxExperts) return 0;
    if (forced >= 1 && forced <= 3) return forced - 1;
    const int64_t rows = a.M / a.E;                       // an expert's rows, on average
    const int64_t panels = a.E * ((a.N + 255) / 256);
    if (rows <= (panels < 128 ? 16 : 6)) return 0;
    if (panels < 128 && (rows + 63) / 64 * (panels < 28 ? 28 : panels) <= 90) return 0;
    return rows >= 128 && panels * ((rows + 255) / 256) >= 256 ? 2 : 1;
}

const char *grouped_kernel_name(const GroupedArgs &a) {
    const int form = grouped_form(a);
    return form == 0   ? "grouped_stream_kernel"
           : form == 1 ? "grouped_gemm_kernel 128-row tiles"
                       : "grouped_gemm_kernel 256-row tiles";
}

hipError_t launch_grouped(int elem, int layout, const GroupedArgs &a, hipStream_t st) {
    if (const int form = grouped_form(a))
        return launch_grouped_gemm(elem, layout, 128 * form, a, st);
    // (e2m1: four tiles a workgroup while that leaves two workgroups a compute unit)
    if (elem == E2M1)
        return a.E * (a.N / 64) >= 512 ? launch_stream<E2M1, ROW32, 4>(a, st)
                                       : launch_stream<E2M1, ROW32, 2>(a, st);
    return layout == ROW32 ? launch_stream<E4M3, ROW32, 2>(a, st)
                           : launch_stream<E4M3, BLK32, 2>(a, st);
}

// ---- staging: the grouped rows' activation in the T16 layout ----
// Row i of the output is source row rows[i] (or i), quantized from bf16 or
// copied from row-major MXFP8 bytes; a source row outside [0, xrows) and the
// rows of the last tile behind offsets[E] are zeros with code 127.  Tiles
// wholly behind offsets[E] are not written (nothing reads them).  One wavefront
// per token tile and quad of 128-K steps, as the T16 quantization
// (mx_quant.hip): lane (r, j) handles 16 values of each half step of token r.
// GIVEN: row-major MXFP8 input, else bf16 quantized by RULE.
template <bool GIVEN, int RULE>
__global__ void __launch_bounds__(256) stage_rows_kernel(StageArgs p, int64_t units) {
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 64;
    if (unit >= units) return;                            // whole wavefronts
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int64_t S = (p.K + 127) / 128, Q = (S + 3) / 4, KB = p.K / 32;
    const int64_t q = unit % Q, mb = unit / Q;
    const int64_t m = 16 * mb + r;
    int64_t end = p.offsets[p.E];
    end = end > p.M ? p.M : end;
    if (16 * mb >= end) return;
    int64_t src = -1;
    if (m < end) src = p.rows ? p.rows[m] : m;
    const bool live = src >= 0 && src < p.xrows;
    uint32_t code[4][2];
    if (GIVEN) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t s = 4 * q + u, k0 = 128 * s + 64 * h + 16 * j;
                const v4u v = live && k0 < p.K
                                  ? *reinterpret_cast<const v4u *>(p.xq + src * p.ldq + k0)
                                  : v4u{0u, 0u, 0u, 0u};
                if (s < S)
                    *reinterpret_cast<v4u *>(p.out + ((mb * S + s) * 2 + h) * 1024 + 16 * lane) = v;
            }
    } else {
        v4u v[4][2][2];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k0 = 128 * (4 * q + u) + 64 * h + 16 * j;
                const bool ok = live && k0 < p.K;
                const uint16_t *at = p.x + (ok ? src * p.ldx + k0 : 0);
                v[u][h][0] = ok ? *reinterpret_cast<const v4u *>(at) : v4u{0u, 0u, 0u, 0u};
                v[u][h][1] = ok ? *reinterpret_cast<const v4u *>(at + 8) : v4u{0u, 0u, 0u, 0u};
            }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t s = 4 * q + u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u o = quant_half_block_cvt<RULE>(v[u][h][0], v[u][h][1], code[u][h]);
                if (s < S)
                    *reinterpret_cast<v4u *>(p.out + ((mb * S + s) * 2 + h) * 1024 + 16 * lane) = o;
            }
        }
    }
    // lane (r, j) writes block 4 s + j's code of four steps; quantized here, it
    // is held by lanes 32 (j % 2) + r and 16 further of half j / 2
    const int from = 32 * (j % 2) + r;
    uint32_t dw = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t blk = 4 * (4 * q + u) + j;
        uint32_t c = 127u;
        if (GIVEN) {
            if (live && blk < KB) c = p.xc[src * p.ldc + blk];
        } else {
            const uint32_t c0 = (uint32_t)__shfl((int)code[u][0], from);
            const uint32_t c1 = (uint32_t)__shfl((int)code[u][1], from);
            if (live && blk < KB) c = j / 2 ? c1 : c0;
        }
        dw |= c << (8 * u);
    }
    reinterpret_cast<uint32_t *>(p.outc)[(mb * Q + q) * 64 + lane] = dw;
}

hipError_t launch_stage_rows(const StageArgs &a, int rule, hipStream_t st) {
    const int64_t Q = ((a.K + 127) / 128 + 3) / 4, units = (a.M + 15) / 16 * Q;
    const dim3 grid((unsigned)((units + 3) / 4)), block(256);
    if (!a.x)
        hipLaunchKernelGGL((stage_rows_kernel<true, RULE_OCP>), grid, block, 0, st, a, units);
    else if (rule == RULE_OCP)
        hipLaunchKernelGGL((stage_rows_kernel<false, RULE_OCP>), grid, block, 0, st, a, units);
    else
        hipLaunchKernelGGL((stage_rows_kernel<false, RULE_CEIL448>), grid, block, 0, st, a, units);
    return hipGetLastError();
}

}  // namespace mx
