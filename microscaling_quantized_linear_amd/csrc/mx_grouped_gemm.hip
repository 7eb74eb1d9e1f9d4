// mx_grouped_gemm.hip -- products grouped by expert, tiled form: the prefill
// GEMM's main loop (mx_gemm.hip) over the row ranges of many experts, with
// e4m3 or e2m1 weights.
//
// Workgroup tile: 256 weight rows of one expert x 128 MT of its rows, four
// wavefronts side by side along the rows; a wavefront owns all 256 weight rows
// and 32 MT rows, 8 x MT output tiles of 32 x 32 accumulated by
// v_mfma_scale_f32_32x32x64_f8f6f4 (A = weights, e4m3 or e2m1; B = e4m3
// activations; per-lane E8M0 scales).
//  - weights: each 128-K step's chunks go straight from memory into one of four
//    LDS buffers, two steps ahead of the matrix cores, one barrier a step;
//  - activations: straight from the T16 layout into registers, a step ahead.  An
//    expert's rows start anywhere in a token tile, so each lane has the offset
//    of its own row; rows past the range read zeros.
//
// Which tile a workgroup takes is decided on the device, where the offsets are:
// the experts' tile counts are added up by a wavefront scan (64 experts at a
// time), so the grid is only an upper bound and the workgroups behind the last
// tile exit.  The tiles are numbered expert by expert, within an expert by
// weight panel, within a panel by row tile; XCD x (of eight, workgroups are
// handed out to them in turn) takes the x-th eighth of that order, so the
// workgroups that run on an XCD together share weight panels and rows in its
// L2.
#include "mx_device.h"
#include "mx_kernels.h"

#include <type_traits>

namespace mx {

typedef __attribute__((address_space(3))) void lds_void;
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kNTW = 8, kGroupedBN = 32 * kNTW;

struct TileAt {
    int e;             // expert, -1: no tile
    int64_t row0, end; // first row of the tile, end of the expert's range
    int tn;            // weight panel
};

// The tile of workgroup bid; every wavefront works it out for itself.
template <int BM>
__device__ inline TileAt find_tile(const GroupedArgs &p, int tiles_n) {
    const int lane = threadIdx.x % 64;
    auto range = [&](int e, int64_t &o0, int64_t &o1) {
        o0 = p.offsets[e];
        o1 = p.offsets[e + 1];
        o0 = o0 < 0 ? 0 : o0;                             // cut to [0, M)
        o1 = o1 > p.M ? p.M : o1;
        return o1 > o0 ? (int)((o1 - o0 + BM - 1) / BM) : 0;
    };
    const int E = (int)p.E;
    // row tiles in all (experts 64 at a time; the first 64 counts are kept)
    int total = 0, first = 0;
    for (int base = 0; base < E; base += 64) {
        int64_t o0, o1;
        int n = base + lane < E ? range(base + lane, o0, o1) : 0;
        if (base == 0) first = n;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
        total += n;
    }
    const int64_t tiles = (int64_t)total * tiles_n, per = (tiles + 7) / 8;
    const int64_t local = blockIdx.x / 8;
    int64_t id = (blockIdx.x % 8) * per + local;
    TileAt at{-1, 0, 0, 0};
    if (local >= per || id >= tiles) return at;
    for (int base = 0; base < E; base += 64) {
        int64_t o0 = 0, o1 = 0;
        const int n = base == 0 ? first : base + lane < E ? range(base + lane, o0, o1) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(inc, o);
            inc += lane >= o ? v : 0;
        }
        const int64_t upto = (int64_t)inc * tiles_n;
        const uint64_t past = __ballot(upto > id);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int cnt = __builtin_amdgcn_readlane(n, l);
            const int before = __builtin_amdgcn_readlane(inc, l) - cnt;
            const int in = (int)(id - (int64_t)before * tiles_n);
            at.e = base + l;
            range(at.e, o0, o1);
            at.tn = in / cnt;
            at.row0 = o0 + (int64_t)(in % cnt) * BM;
            at.end = o1;
            return at;
        }
        id -= (int64_t)__builtin_amdgcn_readlane(inc, 63) * tiles_n;
    }
    return at;
}

__device__ inline float gated(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// MT 32-row slabs a wavefront; TAIL: K % 128 != 0; REM: the step count is not a
// multiple of eight (as in mx_gemm.hip)
template <int ELEM, int LAYOUT, int MT, bool TAIL, bool REM>
__global__ void __launch_bounds__(256, 1) grouped_gemm_kernel(GroupedArgs p) {
    constexpr int NTW = kNTW, BN = kGroupedBN, BM = 128 * MT;
    constexpr int CHUNK = ELEM == E4M3 ? 2048 : 1024;
    constexpr int kCopies = ELEM == E4M3 ? NTW : NTW / 2; // 1 KB copies a wavefront and step
    constexpr int kWBytes = 2 * NTW * CHUNK;
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[kWBytes];
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64) & 3;
    const int S = (int)((p.K + 127) / 128), Q = (S + 3) / 4;
    const int64_t T = p.N / 16;
    const TileAt at = find_tile<BM>(p, (int)((p.N + BN - 1) / BN));
    if (at.e < 0) return;
    // wave-uniform from here on
    const int e = __builtin_amdgcn_readfirstlane(at.e);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(at.tn) * BN;
    const int64_t row0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)at.row0);
    const int64_t end = (uint32_t)__builtin_amdgcn_readfirstlane((int)at.end);
    const int64_t t0 = n0 / 16, mb0 = row0 / 16;

    const int64_t TILEB = 16 * (ELEM == E4M3 ? p.K : p.K / 2);
    const uint32_t tailb = (uint32_t)(TILEB - (int64_t)(S - 1) * CHUNK);
    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(p.w + (e * T + t0) * TILEB, (uint32_t)((T - t0) * TILEB));
    // the rows' token tiles: at most BM / 16 + 1
    const int64_t mleft = (p.M + 15) / 16 - mb0;
    const uint32_t nmb = (uint32_t)(mleft < BM / 16 + 1 ? mleft : BM / 16 + 1);
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(p.xq + mb0 * S * 2048, nmb * (uint32_t)S * 2048u);
    const __amdgpu_buffer_rsrc_t xcr = make_rsrc(p.xct + mb0 * Q * 256, nmb * (uint32_t)Q * 256u);
    const __amdgpu_buffer_rsrc_t cr =
        LAYOUT == ROW32 ? make_rsrc(p.codes + (e * T + t0) * Q * 256, (uint32_t)((T - t0) * Q * 256))
                        : make_rsrc(p.codes + (e * (p.N / 32) + n0 / 32) * Q * 16,
                                    (uint32_t)((p.N / 32 - n0 / 32) * Q * 16));

    // ---- weight copies: unit idx = wave + 4 i lands at idx KB; e4m3: half
    // idx % 2 of tile idx / 2's chunk, e2m1: tile idx's chunk.  Out-of-range
    // offsets get bit 31 (those lanes read zeros). ----
    uint32_t wofs[kCopies], wtail[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int idx = wave + 4 * i;
        const int c = ELEM == E4M3 ? idx / 2 : idx, h = ELEM == E4M3 ? idx % 2 : 0;
        const uint32_t o = (uint32_t)(1024 * h + 16 * lane);
        wofs[i] = t0 + c < T ? (uint32_t)(c * TILEB) + o : kOOB;
        wtail[i] = o >= tailb ? kOOB : 0u;
    }
    auto dma_one = [&](uint8_t *buf, int s, int i) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wr, (lds_void *)(buf + (wave + 4 * i) * 1024), 16,
            (int)((wofs[i] + (uint32_t)s * CHUNK) | (s >= S ? kOOB : 0u) |
                  (TAIL && s == S - 1 ? wtail[i] : 0u)),
            0, 0, 0);
    };

    // ---- operands: lane (g, rr) = lane / 32, lane % 32 holds row rr of a
    // 64-K half step kh.  e4m3: K 16 g .. and 32 + 16 g .., two 16-byte pieces;
    // e2m1: K 32 g .., one 16-byte piece (lane group 2 kh + g of the chunk) ----
    const int rr = lane % 32, g = lane / 32;
    const int off_lane = (rr / 16) * CHUNK + 256 * g + 16 * (rr % 16);
    auto rd = [&](const uint8_t *base, int kh) -> v8i {
        if constexpr (ELEM == E4M3) {
            const uint8_t *cp = base + off_lane + 1024 * kh;
            return cat8(*reinterpret_cast<const v4u *>(cp),
                        *reinterpret_cast<const v4u *>(cp + 512));
        } else {
            const v4u v = *reinterpret_cast<const v4u *>(base + off_lane + 512 * kh);
            return v8i{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
    };
    uint32_t xo[MT], xco[MT];                             // this lane's row of slab mt, or kOOB
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t row = row0 + 32 * MT * wave + 32 * mt + rr;
        const uint32_t mb = (uint32_t)(row / 16 - mb0), slot = (uint32_t)(row % 16);
        xo[mt] = row < end ? mb * (uint32_t)S * 2048u + 256u * g + 16u * slot : kOOB;
        xco[mt] = row < end ? mb * (uint32_t)Q * 256u + 64u * g + 4u * slot : kOOB;
    }
    typedef v8i BFrag[2][MT];                             // [kh][mt]
    constexpr int kB = 4 * MT;                            // activation loads a step
    auto load_b_one = [&](BFrag &b, int s, int n) {       // load n: (kh, mt, piece)
        const int kh = n / (2 * MT), mt = (n / 2) % MT, pc = n % 2;
        const uint32_t u = (xo[mt] + (uint32_t)s * 2048u) | (s >= S ? kOOB : 0u);
        const v4u v = load16(xr, (u + 1024u * kh + 512u * pc) | (u & kOOB));
#pragma unroll
        for (int d = 0; d < 4; ++d) b[kh][mt][4 * pc + d] = (int)v[d];
    };

    struct QScales {
        uint32_t w[NTW][2], x[MT][2];
    };
    const uint32_t clane = (uint32_t)((rr / 16) * Q * 256 + 64 * g + 4 * (rr % 16));
    auto load_qscales = [&](int q, QScales &out) {
        const uint32_t past = q >= Q ? kOOB : 0u;
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
                uint32_t off;
                if (LAYOUT == ROW32)
                    off = clane + (uint32_t)((2 * nt * Q + q) * 256 + 128 * kh);
                else
                    off = 4u * g + (uint32_t)((nt * Q + q) * 16 + 8 * kh);
                out.w[nt][kh] = load4(cr, off | past);
            }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
                const uint32_t u = xco[mt] + (uint32_t)q * 256u + 128u * kh;
                out.x[mt][kh] = load4(xcr, u | (u & kOOB) | past);
            }
    };

    v16f acc[NTW][MT];
    auto step_barrier = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // One 128-K step (the order and its reasons as in mx_gemm.hip): 2 NTW groups
    // (half step kh, weight slab nt) of MT products; the next step's activation
    // loads go out in the first groups, the copies of step s + 2 in the last
    // kCopies; the barrier two groups before the end waits for this wavefront's
    // copies of step s + 1, issued before all of this step's loads.
    constexpr int kMem = kCopies + kB, NG = 2 * NTW;
    auto op_group = [](int i) { return i < kB ? i : i - kB + (NG - kCopies); };
    static_assert(kB <= NG - kCopies && kCopies >= 2, "schedule fits the step");
    static_assert((8 * NG) % 4 == 0 && NG % 4 == 0, "the ring's phase repeats every step");
    v8i af[4];
    auto issue = [&](const uint8_t *buf, int k, int slot) {
        af[slot] = rd(buf + 2 * (k % NTW) * CHUNK, k / NTW);
    };
    auto step = [&](uint8_t *cur, uint8_t *next, uint8_t *ahead, int s, const QScales &sc,
                    BFrag &bc, BFrag &bn, auto uconst, auto firstconst) {
        constexpr int U = decltype(uconst)::value;
        constexpr bool kFirst = decltype(firstconst)::value;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
#pragma unroll
            for (int i = 0; i < kMem; ++i) {
                if (op_group(i) != k) continue;
                if (i < kB) load_b_one(bn, s + 1, i);
                else dma_one(ahead, s + 2, i - kB);
            }
            if (k == NG - 2) {
                static_assert(op_group(kMem - 2) <= NG - 2 && op_group(kMem - 1) == NG - 1,
                              "kMem - 1 loads before the barrier");
                __builtin_amdgcn_s_waitcnt(vmcnt_only(kMem - 1));
                step_barrier();
            }
            if (k + 2 < NG) issue(cur, k + 2, (k + 2) % 4);
            else issue(next, k + 2 - NG, (k + 2) % 4);
            __builtin_amdgcn_sched_barrier(0);
            const int kh = k / NTW, nt = k % NTW;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                acc[nt][mt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    af[k % 4], bc[kh][mt], kFirst && kh == 0 ? v16f{} : acc[nt][mt],
                    ELEM == E4M3 ? 0 : 4, 0, U, (int)sc.w[nt][kh], U, (int)sc.x[mt][kh]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using U0 = std::integral_constant<int, 0>;
    using U1 = std::integral_constant<int, 1>;
    using U2 = std::integral_constant<int, 2>;
    using U3 = std::integral_constant<int, 3>;
    using F0 = std::false_type;

    QScales qa, qb;
    BFrag ba, bb;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) dma_one(lds0, 0, i);
#pragma unroll
    for (int n = 0; n < kB; ++n) load_b_one(ba, 0, n);
    load_qscales(0, qa);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) dma_one(lds1, 1, i);
    __builtin_amdgcn_s_waitcnt(vmcnt_only(kCopies));
    __syncthreads();
    issue(lds0, 0, 0);
    issue(lds0, 1, 1);
    const int S8 = REM ? S / 8 * 8 : S;
    for (int s = 0; s < S8; s += 8) {
        const int q = s / 4;
        load_qscales(q + 1, qb);
        if (s == 0)
            step(lds0, lds1, lds2, s + 0, qa, ba, bb, U0{}, std::true_type{});
        else
            step(lds0, lds1, lds2, s + 0, qa, ba, bb, U0{}, F0{});
        step(lds1, lds2, lds3, s + 1, qa, bb, ba, U1{}, F0{});
        step(lds2, lds3, lds0, s + 2, qa, ba, bb, U2{}, F0{});
        step(lds3, lds0, lds1, s + 3, qa, bb, ba, U3{}, F0{});
        load_qscales(q + 2, qa);
        step(lds0, lds1, lds2, s + 4, qb, ba, bb, U0{}, F0{});
        step(lds1, lds2, lds3, s + 5, qb, bb, ba, U1{}, F0{});
        step(lds2, lds3, lds0, s + 6, qb, ba, bb, U2{}, F0{});
        step(lds3, lds0, lds1, s + 7, qb, bb, ba, U3{}, F0{});
    }
    // REM: the last S % 8 steps in nested uniform conditions
    if (REM && S8 < S) {
        const int s = S8, q = s / 4;
        if (s == 0) {
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[nt][mt] = v16f{};
        }
        load_qscales(q + 1, qb);
        step(lds0, lds1, lds2, s + 0, qa, ba, bb, U0{}, F0{});
        if (s + 1 < S) {
            step(lds1, lds2, lds3, s + 1, qa, bb, ba, U1{}, F0{});
            if (s + 2 < S) {
                step(lds2, lds3, lds0, s + 2, qa, ba, bb, U2{}, F0{});
                if (s + 3 < S) {
                    step(lds3, lds0, lds1, s + 3, qa, bb, ba, U3{}, F0{});
                    if (s + 4 < S) {
                        step(lds0, lds1, lds2, s + 4, qb, ba, bb, U0{}, F0{});
                        if (s + 5 < S) {
                            step(lds1, lds2, lds3, s + 5, qb, bb, ba, U1{}, F0{});
                            if (s + 6 < S)
                                step(lds2, lds3, lds0, s + 6, qb, ba, bb, U2{}, F0{});
                        }
                    }
                }
            }
        }
    }

    // the copies of zeros behind the last step have landed too: none outlives
    // the workgroup
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));

    // ---- epilogue: element i of lane (g, rr) in tile (nt, mt) is weight row
    // 32 nt + 8 (i / 4) + 4 g + i % 4 and row 32 mt + rr.  Pairs are rounded
    // together, v_permlane32_swap trades pieces between lanes rr and rr + 32,
    // and every lane stores 16 bytes; what lies past the range or N is dropped
    // by its out-of-range offset. ----
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    auto pk = [](float lo, float hi) -> uint32_t {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
    };
    const int64_t rows = end - row0 < BM ? end - row0 : BM;
    const int64_t width = p.epi ? p.N / 2 : p.N;
    const __amdgpu_buffer_rsrc_t yr =
        make_rsrc(p.y + row0 * p.ldy, (uint32_t)(((rows - 1) * p.ldy + width) * 2));
    uint32_t ybase[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int row = 32 * MT * wave + 32 * mt + rr;
        ybase[mt] = row < rows ? (uint32_t)(row * p.ldy * 2) : kOOB;
    }
    const int64_t nlim = p.N - n0;                        // weight rows left
#pragma unroll
    for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const v16f &c = acc[nt][mt];
            if (p.epi) {
                // pair of rows 2 i, 2 i + 1 -> column i: dword 2 a + g of the
                // slab's eight holds columns 4 a + 2 g, + 1
                uint32_t d[4];
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    d[a] = pk(gated(c[4 * a], c[4 * a + 1]), gated(c[4 * a + 2], c[4 * a + 3]));
                const auto s02 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
                const auto s13 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
                const uint32_t col = (uint32_t)(n0 / 2) + 16u * nt + 8u * g;
                const bool in = 32 * nt + 16 * g < nlim;
                __builtin_amdgcn_raw_buffer_store_b128(
                    v4u{s02[0], s02[1], s13[0], s13[1]}, yr,
                    (int)(in ? ybase[mt] + 2u * col : kOOB), 0, 0);
            } else {
#pragma unroll
                for (int a0 = 0; a0 < 4; a0 += 2) {
                    uint32_t o[2][2];
#pragma unroll
                    for (int d = 0; d < 2; ++d)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 4 * (a0 + d) + 2 * h;
                            o[d][h] = pk(c[i], c[i + 1]);
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const auto sw =
                            __builtin_amdgcn_permlane32_swap(o[0][h], o[1][h], false, false);
                        o[0][h] = sw[0];
                        o[1][h] = sw[1];
                    }
                    const uint32_t col = (uint32_t)n0 + 32u * nt + 8u * (a0 + g);
                    const bool in = 32 * nt + 8 * (a0 + g) < nlim;
                    __builtin_amdgcn_raw_buffer_store_b128(
                        v4u{o[0][0], o[0][1], o[1][0], o[1][1]}, yr,
                        (int)(in ? ybase[mt] + 2u * col : kOOB), 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);                // one slab's values at a time
    }
}

template <int ELEM, int LAYOUT, int MT>
static hipError_t launch_mt(const GroupedArgs &a, hipStream_t st) {
    constexpr int64_t BM = 128 * MT;
    const int64_t tiles_n = (a.N + kGroupedBN - 1) / kGroupedBN;
    // ceil over the experts: at most (M + E (BM - 1)) / BM row tiles, and at
    // most one more than the whole tiles for every expert with a row
    int64_t rows = (a.M + a.E * (BM - 1)) / BM;
    if (rows > a.M) rows = a.M;
    const int64_t tiles = (rows * tiles_n + 7) / 8 * 8;   // whole eighths
    const dim3 grid((unsigned)tiles), block(256);
    const bool tail = a.K % 128 != 0, rem = (a.K + 127) / 128 % 8 != 0;
    if (tail)
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, MT, true, true>), grid, block, 0, st, a);
    else if (rem)
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, MT, false, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, MT, false, false>), grid, block, 0, st, a);
    return hipGetLastError();
}

hipError_t launch_grouped_gemm(int elem, int layout, int mt, const GroupedArgs &a,
                               hipStream_t st) {
    if (elem == E2M1)
        return mt == 1 ? launch_mt<E2M1, ROW32, 1>(a, st) : launch_mt<E2M1, ROW32, 2>(a, st);
    if (layout == ROW32)
        return mt == 1 ? launch_mt<E4M3, ROW32, 1>(a, st) : launch_mt<E4M3, ROW32, 2>(a, st);
    return mt == 1 ? launch_mt<E4M3, BLK32, 1>(a, st) : launch_mt<E4M3, BLK32, 2>(a, st);
}

}  // namespace mx
