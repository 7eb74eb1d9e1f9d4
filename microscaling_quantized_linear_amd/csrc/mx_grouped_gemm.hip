// mx_grouped_gemm.hip -- products grouped by expert, tiled form: the prefill
// GEMM's main loop (mx_gemm.hip) over the row ranges of many experts, with
// e4m3 or e2m1 weights.
//
// A tile is 256 weight rows of one expert x up to 256 (large) or 128 (small) of
// its rows, for a workgroup of four wavefronts.  32 x 32 output tiles are
// accumulated by v_mfma_scale_f32_32x32x64_f8f6f4 (A = weights, e4m3 or e2m1;
// B = e4m3 activations; per-lane E8M0 scales).  In a large tile each wavefront
// owns all 256 weight rows and 64 rows; in a small one the wavefronts stand two
// by two, 128 weight rows and 64 rows each: with four side by side each reads
// all the weights' 32 KB from LDS a step, as long as its products take.
//  - weights: each 128-K step's chunks go straight from memory into one of four
//    LDS buffers, two steps ahead of the matrix cores, one barrier a step;
//  - activations: straight from the T16 layout into registers, a step ahead.  An
//    expert's rows start anywhere in a token tile, so each lane has the offset
//    of its own row; rows past the range read zeros.
//
// The tiles are found on the device, where the offsets are: every workgroup adds
// up the experts' tiles once (a wavefront scan, 64 experts at a time, kept in
// LDS).  An expert's rows make large tiles and, for a remainder of up to 128
// rows, a small one.  The large tiles of all experts come first, then the small
// ones, each expert by expert, within an expert by weight panel, within a panel
// by row tile; XCD x (of eight, workgroups are handed out to them in turn) takes
// the x-th eighth of either list, and its workgroups take its tiles in turn, so
// that those running together share weight panels and rows in its L2, and the
// half-length tiles even out the end.
// One workgroup stays on each compute unit: the next tile's first loads are
// issued ahead of the stores of the last one, which hides their latency (a tile
// of K = 2048 takes 17 us of products; a launch a tile cost 4 us more).
#include "mx_device.h"
#include "mx_kernels.h"

#include <type_traits>

namespace mx {

typedef __attribute__((address_space(3))) void lds_void;
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kGroupedBN = 256;            // weight rows of a tile
constexpr int kUnits = 256;                // compute units, one workgroup each

struct TileAt {
    int e;             // expert, -1: no tile
    int row0, end;     // first row of the tile, end of the expert's range
    int tn;            // weight panel
};

__device__ inline float gated(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// TAIL: K % 128 != 0; REM: the step count is not a multiple of eight (as in
// mx_gemm.hip).  bm: rows of a tile at most, 256 or 128 (then all are small).
template <int ELEM, int LAYOUT, bool EPI, bool TAIL, bool REM>
__global__ void __launch_bounds__(256, 1) grouped_gemm_kernel(GroupedArgs p, int bm) {
    constexpr int BN = kGroupedBN;
    constexpr int CHUNK = ELEM == E4M3 ? 2048 : 1024;
    constexpr int kCopies = ELEM == E4M3 ? 8 : 4;         // 1 KB copies a wavefront and step
    constexpr int kWBytes = 16 * CHUNK;
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[kWBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[kWBytes];
    __shared__ int upto[2][kGroupedMaxExperts];           // large, small tiles up to expert e
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64) & 3;
    const int64_t T = p.N / 16;
    const int E = (int)p.E, tiles_n = (int)((p.N + BN - 1) / BN);

    // ---- the tiles: large[e] = whole bm rows (and a remainder above 128), small[e] =
    // a remainder of up to 128 rows (bm = 128: all of them are small) ----
    auto range = [&](int e, int &o0, int &o1) {           // cut to [0, M)
        o0 = p.offsets[e];
        o1 = p.offsets[e + 1];
        o0 = o0 < 0 ? 0 : o0;
        o1 = o1 > (int)p.M ? (int)p.M : o1;
        o1 = o1 < o0 ? o0 : o1;
    };
    auto large_of = [&](int rows) { return bm == 256 ? rows / 256 + (rows % 256 > 128) : 0; };
    auto small_of = [&](int rows) {
        return bm == 256 ? (rows % 256 > 0 && rows % 256 <= 128) : (rows + 127) / 128;
    };
    if (wave == 0) {
        int large = 0, small = 0;
        for (int base = 0; base < E; base += 64) {
            int n[2] = {0, 0};
            if (base + lane < E) {
                int o0, o1;
                range(base + lane, o0, o1);
                n[0] = large_of(o1 - o0);
                n[1] = small_of(o1 - o0);
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int v = __shfl_up(n[k], o);
                    n[k] += lane >= o ? v : 0;
                }
            if (base + lane < E) {
                upto[0][base + lane] = large + n[0];
                upto[1][base + lane] = small + n[1];
            }
            large += __builtin_amdgcn_readlane(n[0], 63);
            small += __builtin_amdgcn_readlane(n[1], 63);
        }
    }
    __syncthreads();
    // (offsets that descend could claim more tiles than M rows have: not served)
    if (upto[0][E - 1] + upto[1][E - 1] > (int)(p.M / 128) + E) return;
    // this XCD's parts of the two lists
    const int xcd = blockIdx.x % 8;
    const int all[2] = {__builtin_amdgcn_readfirstlane(upto[0][E - 1]) * tiles_n,
                        __builtin_amdgcn_readfirstlane(upto[1][E - 1]) * tiles_n};
    int from[2], count[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int per = (all[k] + 7) / 8;
        from[k] = xcd * per;
        const int left = all[k] - from[k];
        count[k] = left < 0 ? 0 : left < per ? left : per;
    }
    // tile number i of this XCD
    auto find = [&](int i) {
        TileAt at{-1, 0, 0, 0};
        if (i >= count[0] + count[1]) return at;
        const int k = i < count[0] ? 0 : 1;
        const int id = from[k] + (k ? i - count[0] : i);
        const int unit = id / tiles_n;                    // the row tile, counted over the experts
        int e = 0, before = 0, cnt = 0;
        for (int base = 0; base < E; base += 64) {
            const int at_e = base + lane < E ? upto[k][base + lane] : 0x7fffffff;
            const uint64_t past = __ballot(at_e > unit);
            if (past) {
                e = base + __builtin_ctzll(past);
                break;
            }
        }
        before = e ? __builtin_amdgcn_readfirstlane(upto[k][e - 1]) : 0;
        cnt = __builtin_amdgcn_readfirstlane(upto[k][e]) - before;
        const int in = id - before * tiles_n;
        int o0, o1;
        range(e, o0, o1);
        at.e = e;
        at.tn = in / cnt;
        at.row0 = o0 + (k && bm == 256 ? (o1 - o0) / 256 * 256 : in % cnt * (k ? 128 : 256));
        at.end = o1;
        at.e = __builtin_amdgcn_readfirstlane(at.e);
        at.tn = __builtin_amdgcn_readfirstlane(at.tn);
        at.row0 = __builtin_amdgcn_readfirstlane(at.row0);
        at.end = __builtin_amdgcn_readfirstlane(at.end);
        return at;
    };

    // One tile: its first activations and scales, the products, the next tile's
    // first copies, then the stores.  Ahead of the copies a barrier: every
    // wavefront is past its last read of the weight buffers (the copies of zeros
    // behind a tile's last step land in order before the new ones).
    int i = blockIdx.x / 8;
    TileAt at = find(i);
    if (at.e < 0) return;
    bool small = i >= count[0];
    bool fresh = true;                                    // the tile's first copies are not out yet
    do {
        // Opaque copies of the lane and the step count: what is worked out from them
        // would otherwise be kept over the whole loop, beyond the registers.
        int lane_now = lane, steps_now = (int)((p.K + 127) / 128);
        asm volatile("" : "+v"(lane_now));
        asm volatile("" : "+s"(steps_now));
        const int lane = lane_now, S = steps_now, Q = (S + 3) / 4;
        // ---- a tile's addresses ----
        const int64_t TILEB = 16 * (ELEM == E4M3 ? p.K : p.K / 2);
        const uint32_t tailb = (uint32_t)(TILEB - (int64_t)(S - 1) * CHUNK);
        const int rr = lane % 32, g = lane / 32;
        __amdgpu_buffer_rsrc_t wr, xr, xcr, cr;
        int slab0 = 0;                                    // this wavefront's first weight slab
        uint32_t xo[2], xco[2];                           // this lane's row of slab mt, or kOOB
        auto weights = [&](const TileAt &at) {
            const int64_t t0 = (int64_t)at.tn * (BN / 16);
            const int64_t panel_tiles = T - t0 < BN / 16 ? T - t0 : BN / 16;
            wr = make_rsrc(p.w + (at.e * T + t0) * TILEB, (uint32_t)(panel_tiles * TILEB));
        };
        auto setup = [&](const TileAt &at, bool small) {
            const int64_t t0 = (int64_t)at.tn * (BN / 16), mb0 = at.row0 / 16;
            const int64_t e = at.e;
            const int64_t panel_tiles = T - t0 < BN / 16 ? T - t0 : BN / 16;
            weights(at);
            // the rows' token tiles: at most 17
            const int64_t mleft = (p.M + 15) / 16 - mb0;
            const uint32_t nmb = (uint32_t)(mleft < 17 ? mleft : 17);
            xr = make_rsrc(p.xq + mb0 * S * 2048, nmb * (uint32_t)S * 2048u);
            xcr = make_rsrc(p.xct + mb0 * Q * 256, nmb * (uint32_t)Q * 256u);
            cr = LAYOUT == ROW32
                     ? make_rsrc(p.codes + (e * T + t0) * Q * 256,
                                 (uint32_t)(panel_tiles * Q * 256))
                     : make_rsrc(p.codes + (e * (p.N / 32) + t0 / 2) * Q * 16,
                                 (uint32_t)(panel_tiles / 2 * Q * 16));
            slab0 = small ? wave / 2 * 4 : 0;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const int row = at.row0 + 64 * (small ? wave % 2 : wave) + 32 * mt + rr;
                const uint32_t mb = (uint32_t)(row / 16 - (int)mb0), slot = (uint32_t)(row % 16);
                xo[mt] = row < at.end ? mb * (uint32_t)S * 2048u + 256u * g + 16u * slot : kOOB;
                xco[mt] = row < at.end ? mb * (uint32_t)Q * 256u + 64u * g + 4u * slot : kOOB;
            }
        };

        // ---- weight copies: unit idx = wave + 4 i lands at idx KB; e4m3: half
        // idx % 2 of tile idx / 2's chunk, e2m1: tile idx's chunk.  Out-of-range
        // offsets (steps past S, a cut last chunk, tiles past the panel through the
        // resource's end) read zeros. ----
        // (e4m3: wave and i give half wave % 2 of tile 2 i + wave / 2)
        const uint32_t wlane = (ELEM == E4M3 ? 1024u * (wave % 2) : 0u) + 16u * lane;
        const uint32_t wtail = TAIL && wlane >= tailb ? kOOB : 0u;
        auto dma_one = [&](uint8_t *buf, int s, int i) {
            const int c = ELEM == E4M3 ? 2 * i + wave / 2 : 4 * i + wave;
            const uint32_t bad = (s >= S ? kOOB : 0u) | (TAIL && s == S - 1 ? wtail : 0u);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                wr, (lds_void *)(buf + (wave + 4 * i) * 1024), 16,
                (int)((wlane + (uint32_t)(c * TILEB + (int64_t)s * CHUNK)) | bad), 0, 0, 0);
        };

        // ---- operands: lane (g, rr) = lane / 32, lane % 32 holds row rr of a
        // 64-K half step kh.  e4m3: K 16 g .. and 32 + 16 g .., two 16-byte pieces;
        // e2m1: K 32 g .., one 16-byte piece (lane group 2 kh + g of the chunk) ----
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
        typedef v8i BFrag[2][2];                              // [kh][mt]
        constexpr int kB = 8;                                 // activation loads a step
        auto load_b_one = [&](BFrag &b, int s, int n) {       // load n: (kh, mt, piece)
            const int kh = n / 4, mt = (n / 2) % 2, pc = n % 2;
            const uint32_t u = (xo[mt] + (uint32_t)s * 2048u) | (s >= S ? kOOB : 0u);
            const v4u v = load16(xr, (u + 1024u * kh + 512u * pc) | (u & kOOB));
#pragma unroll
            for (int d = 0; d < 4; ++d) b[kh][mt][4 * pc + d] = (int)v[d];
        };
        // the scale dwords of a quad of steps: slab i of the wavefront and the rows
        struct QScales {
            uint32_t w[8][2], x[2][2];
        };
        const uint32_t clane = (uint32_t)((rr / 16) * Q * 256 + 64 * g + 4 * (rr % 16));
        auto load_qscales = [&](int q, QScales &out, auto slabs) {
            const uint32_t past = q >= Q ? kOOB : 0u;
#pragma unroll
            for (int nt = 0; nt < decltype(slabs)::value; ++nt)
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    uint32_t off;
                    if (LAYOUT == ROW32)
                        off = clane + (uint32_t)((2 * (slab0 + nt) * Q + q) * 256 + 128 * kh);
                    else
                        off = 4u * g + (uint32_t)(((slab0 + nt) * Q + q) * 16 + 8 * kh);
                    out.w[nt][kh] = load4(cr, off | past);
                }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    const uint32_t u = xco[mt] + (uint32_t)q * 256u + 128u * kh;
                    out.x[mt][kh] = load4(xcr, u | (u & kOOB) | past);
                }
        };
        using U0 = std::integral_constant<int, 0>;
        using U1 = std::integral_constant<int, 1>;
        using U2 = std::integral_constant<int, 2>;
        using U3 = std::integral_constant<int, 3>;
        using F0 = std::false_type;
        using Slabs8 = std::integral_constant<int, 8>;
        using Slabs4 = std::integral_constant<int, 4>;

        auto step_barrier = [] {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        BFrag ba, bb;
        QScales qa, qb;
        // a tile's first copies
        auto begin = [&] {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) dma_one(lds0, 0, i);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) dma_one(lds1, 1, i);
        };

        // ---- the products of a tile: NW weight slabs x 2 row slabs a wavefront ----
        auto products = [&](auto slabs, v16f (&acc)[decltype(slabs)::value][2]) {
            constexpr int NW = decltype(slabs)::value, NG = 2 * NW;
            // One 128-K step (the order and its reasons as in mx_gemm.hip): NG groups
            // (half step kh, weight slab nt) of two products.  Spread over the groups
            // go out the next step's activation loads, then the copies of step s + 2.
            // The barrier two groups before the end waits for this wavefront's copies
            // of step s + 1, issued before all of this step's loads.
            constexpr int kMem = kCopies + kB;
            auto op_group = [](int i) { return i * NG / kMem; };
            constexpr int kBefore = [] {                      // loads of groups 0 .. NG - 2
                int n = 0;
                for (int i = 0; i < kMem; ++i) n += i * NG / kMem <= NG - 2;
                return n;
            }();
            static_assert(NG % 4 == 0, "the ring's phase repeats every step");
            v8i af[4];
            auto issue = [&](const uint8_t *buf, int k, int slot) {
                af[slot] = rd(buf + 2 * (slab0 + k % NW) * CHUNK, k / NW);
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
                        __builtin_amdgcn_s_waitcnt(vmcnt_only(kBefore));
                        step_barrier();
                    }
                    if (k + 2 < NG) issue(cur, k + 2, (k + 2) % 4);
                    else issue(next, k + 2 - NG, (k + 2) % 4);
                    __builtin_amdgcn_sched_barrier(0);
                    const int kh = k / NW, nt = k % NW;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
                        acc[nt][mt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            af[k % 4], bc[kh][mt], kFirst && kh == 0 ? v16f{} : acc[nt][mt],
                            ELEM == E4M3 ? 0 : 4, 0, U, (int)sc.w[nt][kh], U, (int)sc.x[mt][kh]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            issue(lds0, 0, 0);
            issue(lds0, 1, 1);
            const int S8 = REM ? S / 8 * 8 : S;
            for (int s = 0; s < S8; s += 8) {
                const int q = s / 4;
                load_qscales(q + 1, qb, slabs);
                if (s == 0)
                    step(lds0, lds1, lds2, s + 0, qa, ba, bb, U0{}, std::true_type{});
                else
                    step(lds0, lds1, lds2, s + 0, qa, ba, bb, U0{}, F0{});
                step(lds1, lds2, lds3, s + 1, qa, bb, ba, U1{}, F0{});
                step(lds2, lds3, lds0, s + 2, qa, ba, bb, U2{}, F0{});
                step(lds3, lds0, lds1, s + 3, qa, bb, ba, U3{}, F0{});
                load_qscales(q + 2, qa, slabs);
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
                    for (int nt = 0; nt < NW; ++nt)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) acc[nt][mt] = v16f{};
                }
                load_qscales(q + 1, qb, slabs);
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
        };

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
        auto store = [&](const TileAt &at, int first, auto slabs, bool small,
                         const v16f (&acc)[decltype(slabs)::value][2]) {
            constexpr int NW = decltype(slabs)::value;
            const int most = small ? 128 : 256;
            const int rows = at.end - at.row0 < most ? at.end - at.row0 : most;
            const int64_t width = EPI ? p.N / 2 : p.N;
            const __amdgpu_buffer_rsrc_t yr = make_rsrc(
                p.y + (int64_t)at.row0 * p.ldy, (uint32_t)(((rows - 1) * p.ldy + width) * 2));
            const int n0 = at.tn * BN + 32 * first;           // this wavefront's first weight row
            uint32_t ybase[2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const int row = 64 * (small ? wave % 2 : wave) + 32 * mt + rr;
                ybase[mt] = row < rows ? (uint32_t)(row * p.ldy * 2) : kOOB;
            }
            const int nlim = (int)p.N - n0;                   // weight rows left
#pragma unroll
            for (int nt = 0; nt < NW; ++nt) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const v16f &c = acc[nt][mt];
                    if constexpr (EPI) {
                        // pair of rows 2 i, 2 i + 1 -> column i: dword 2 a + g of the
                        // slab's eight holds columns 4 a + 2 g, + 1
                        uint32_t d[4];
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            d[a] = pk(gated(c[4 * a], c[4 * a + 1]),
                                      gated(c[4 * a + 2], c[4 * a + 3]));
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
                                const auto sw = __builtin_amdgcn_permlane32_swap(
                                    o[0][h], o[1][h], false, false);
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
                __builtin_amdgcn_sched_barrier(0);            // one slab's values at a time
            }
        };

        i += gridDim.x / 8;
        const TileAt after = find(i);
        setup(at, small);
        if (fresh) begin();
        fresh = false;
        auto tile = [&](auto slabs, auto smallconst) {
#pragma unroll
            for (int n = 0; n < kB; ++n) load_b_one(ba, 0, n);
            load_qscales(0, qa, slabs);
            // these, and with them the older copies, have landed
            __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
            step_barrier();
            v16f acc[decltype(slabs)::value][2];
            products(slabs, acc);
            step_barrier();
            if (after.e >= 0) {
                weights(after);
                begin();
            }
            __builtin_amdgcn_sched_barrier(0);
            store(at, slab0, slabs, decltype(smallconst)::value, acc);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (small) tile(Slabs4{}, std::true_type{});
        else tile(Slabs8{}, std::false_type{});
        at = after;
        small = i >= count[0];
    } while (at.e >= 0);
    // nothing outlives the workgroup
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
}

template <int ELEM, int LAYOUT, bool EPI>
static hipError_t launch_epi(int bm, const GroupedArgs &a, hipStream_t st) {
    const int64_t tiles_n = (a.N + kGroupedBN - 1) / kGroupedBN;
    // at most one tile per started 128 rows of an expert
    int64_t rows = (a.M + 127) / 128 + a.E;
    if (rows > a.M) rows = a.M;
    int64_t grid = (rows * tiles_n + 7) / 8 * 8;          // all eight XCDs
    if (grid > kUnits) grid = kUnits;
    const dim3 blocks((unsigned)grid), threads(256);
    const bool tail = a.K % 128 != 0, rem = (a.K + 127) / 128 % 8 != 0;
    if (tail)
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, EPI, true, true>), blocks, threads, 0, st,
                           a, bm);
    else if (rem)
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, EPI, false, true>), blocks, threads, 0, st,
                           a, bm);
    else
        hipLaunchKernelGGL((grouped_gemm_kernel<ELEM, LAYOUT, EPI, false, false>), blocks, threads, 0, st,
                           a, bm);
    return hipGetLastError();
}

template <int ELEM, int LAYOUT>
static hipError_t launch_layout(int bm, const GroupedArgs &a, hipStream_t st) {
    return a.epi ? launch_epi<ELEM, LAYOUT, true>(bm, a, st)
                 : launch_epi<ELEM, LAYOUT, false>(bm, a, st);
}

hipError_t launch_grouped_gemm(int elem, int layout, int bm, const GroupedArgs &a,
                               hipStream_t st) {
    if (elem == E2M1) return launch_layout<E2M1, ROW32>(bm, a, st);
    return layout == ROW32 ? launch_layout<E4M3, ROW32>(bm, a, st)
                           : launch_layout<E4M3, BLK32>(bm, a, st);
}

}  // namespace mx
