// mx_lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   v[m][r] = scale[g] * sum_k x[m][k] A[g][r][k],       g = ids[m]
//   y[m][n] = bf16(base[m][n] + sum_r v[m][r] B[g][n][r])
// and y[m] = base[m] where ids[m] names no adapter.
//
// Two launches.  Both cut the rows into tiles of 16 MT rows and walk the
// distinct adapters among a tile's ids (the first lane of each, by ballots), so
// rows need no order: a tile of one prompt meets one adapter, a tile of 16
// decoding requests up to 16, and each adapter's matrix is read once a tile.
// The adapters of a tile can be shared out over several workgroups.
//   shrink  v in bf16 matrix-core products (16 x 16 x 32, adapter rows x
//           tokens), K split over workgroups and, in each, over eight
//           wavefronts; the partial sums stay in fp32 in the workspace, added
//           in a fixed order.
//   expand  v as the sum of two bf16 numbers (its first eight significant bits
//           and the remainder's rounding, 16 in all), each with a product of its
//           own against the same registers of B: v loses nothing that the bf16
//           result would show, and B is read once.  Cut rather than rounded, the
//           first number leaves a remainder of its own sign: where its products
//           overflow, the remainder's cannot be the opposite infinity.  The
//           projection is added in fp32 and y rounded once.
// Bounds: at decode the adapters' bytes, 2 R (N + K) each, and two launches'
// latency; at prefill x, base and y, 2 K + 4 N bytes a row.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int kShrinkWaves = 8;
constexpr int kUnits = 8;                  // units of 32 values of K a wavefront (few rows)
// Wavefronts of an expand workgroup, 128 columns each (two row groups in a
// 64-row tile).  Many rows: eight, so that v is staged once for 512 columns and
// two workgroups fill a compute unit's registers and LDS.  Few rows: two, for
// more workgroups.
constexpr int expand_waves(int mt) { return mt == 4 ? 8 : 2; }

// Rows of a tile, in units of 16: 64-row tiles read an adapter's matrices a
// quarter as often, 16-row tiles give four times the workgroups.
static int lora_mt(int64_t M, bool invariant) { return M >= 512 && !invariant ? 4 : 1; }
static int64_t lora_tiles(int64_t M, int mt) { return (M + 16 * mt - 1) / (16 * mt); }
// K splits of the shrink.  Few rows: eight units for each of eight wavefronts.
// Many rows: about a workgroup a compute unit, of at least 1024 values of K:
// every split's partial sums are read again by all of the expand's column groups.
int64_t lora_splits(int64_t M, int64_t K, bool invariant) {
    if (lora_mt(M, invariant) == 1) {
        const int64_t per = 32 * kUnits * kShrinkWaves;
        return (K + per - 1) / per;
    }
    const int64_t most = (K + 1023) / 1024, tiles = lora_tiles(M, 4);
    const int64_t want = (256 + tiles - 1) / tiles;
    return want < most ? want : most;
}
// Workgroups that share a tile's adapters, up to `target` in all: a decode
// step's rows may all differ, and a tile where two prompts meet would otherwise
// take twice as long as the rest; those left without an adapter end at once.
static int lora_shares(int64_t M, int mt, int64_t groups, int64_t target) {
    const int64_t most = 16 * mt, want = (target + groups - 1) / groups;
    const int64_t g = want < most ? want : most;
    return (int)(g < M ? g : M);
}

// The 64-row tile of workgroup x, -1 behind the last: XCD i (of eight,
// workgroups go to them in turn) takes the i-th eighth of the tiles, so that
// neighbouring tiles, which mostly share an adapter, find it in one L2.
__device__ inline int64_t tile_of(const LoraArgs &p, int64_t x) {
    const int64_t tiles = (p.M + 63) / 64, per = (tiles + 7) / 8;
    const int64_t t = x % 8 * per + x / 8;
    return t < tiles ? t : -1;
}
static int64_t grid_tiles(int64_t M, int mt) {
    const int64_t t = lora_tiles(M, mt);
    return mt == 4 ? (t + 7) / 8 * 8 : t;
}

// Calls f(adapter, mask of its rows) for the tile's distinct adapters number
// share, share + shares, ...; returns the mask of rows with an adapter.
template <class F>
__device__ inline uint64_t each_adapter(const LoraArgs &p, int64_t m0, int rows, int share,
                                        int shares, F f) {
    const int lane = threadIdx.x % 64;
    int id = -1;
    if (lane < rows && m0 + lane < p.M) id = p.ids[m0 + lane];
    const bool valid = id >= 0 && id < (int)p.L;
    const uint64_t all = __ballot(valid);
    uint64_t todo = all;
    for (int n = 0; todo; ++n) {
        const int key = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t same = __ballot(valid && id == key);
        todo &= ~same;
        if (n % shares == share) f(key, same);
    }
    return all;
}

// Few rows (one 16-row tile): operands straight from memory.
template <int RT>
__global__ void __launch_bounds__(64 * kShrinkWaves) lora_shrink_kernel(LoraArgs p, int splits,
                                                                        int shares) {
    __shared__ v4f red[kShrinkWaves][64];
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int split = blockIdx.y % splits, rank0 = blockIdx.y / splits * (16 * RT);
    const int share = blockIdx.z;
    const int64_t Rp = (p.R + 15) / 16 * 16;
    // this wavefront's units of 32 values of K
    const int units = (int)(p.K / 32), parts = splits * kShrinkWaves;
    const int part = split * kShrinkWaves + wave;
    const int u0 = (int)((int64_t)units * part / parts);
    const int u1 = (int)((int64_t)units * (part + 1) / parts);
    const int64_t left = p.M - m0 < 16 ? p.M - m0 : 16;
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(p.x + m0 * p.ldx, (uint32_t)(((left - 1) * p.ldx + p.K) * 2));
    const uint32_t row_bytes = (uint32_t)(p.K * 2);

    each_adapter(p, m0, 16, share, shares, [&](int g, uint64_t same) {
        const __amdgpu_buffer_rsrc_t ar =
            make_rsrc(p.a + (int64_t)g * p.R * p.K, (uint32_t)(p.R * p.K * 2));
        const uint32_t xo = same >> r & 1 ? (uint32_t)(r * p.ldx * 2) : kOOB;
        uint32_t ao[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int rank = rank0 + 16 * t + r;
            ao[t] = rank < p.R ? (uint32_t)rank * row_bytes : kOOB;
        }
        v4f acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
        // P units a batch, in straight line so that each batch's loads are out
        // ahead of the products of the one before; a unit past the wavefront's
        // range reads zeros
        constexpr int P = RT >= 4 ? 4 : 8;
        constexpr int NB = kUnits / P;
        v4u av[2][P][RT], xv[2][P];
        auto load = [&](int n, int u) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const uint32_t k = 64u * (uint32_t)(u + q) + 16u * j;
                const uint32_t past = u + q < u1 ? 0u : kOOB;
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    av[n][q][t] = load16(ar, ((ao[t] & ~kOOB) + k) | (ao[t] & kOOB) | past);
                xv[n][q] = load16(xr, ((xo & ~kOOB) + k) | (xo & kOOB) | past);
            }
        };
        load(0, u0);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (n + 1 < NB) load((n + 1) % 2, u0 + P * (n + 1));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t] = mfma_bf16(as_bf16x8(av[n % 2][q][t]), as_bf16x8(xv[n % 2][q]),
                                       acc[t]);
            __builtin_amdgcn_sched_barrier(0);
        }
        // element i of lane (j, r): rank 4 j + i, token r of each 16 x 16 tile
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            red[wave][lane] = acc[t];
            __syncthreads();
            if (wave == 0) {
                v4f s = red[0][lane];
#pragma unroll
                for (int w = 1; w < kShrinkWaves; ++w) s += red[w][lane];
                const int rank = rank0 + 16 * t + 4 * j;
                if ((same >> r & 1) && rank < Rp)
                    *reinterpret_cast<v4f *>(p.ws + ((int64_t)split * p.M + m0 + r) * Rp + rank) =
                        s;
            }
            __syncthreads();
        }
    });
}

// Many rows: 64-row tiles, one 16-row slab a wavefront, so no sum crosses
// wavefronts.  K goes in steps of 64 values (128 bytes, a whole line of each
// row): x and A are copied straight into LDS three steps ahead, eight rows and
// 1 KB a copy, because operand-shaped loads (64 bytes of 16 rows) reach memory
// as half lines: x alone then streamed at 2.6 TB/s.  x and, in the expand, the
// projection go past the caches (22 -> 20 and 31 -> 27 us at M = 4096, K = 7168,
// R = 64, N = 4096).  Piece c of a row's eight 16-byte pieces stands at
// c ^ row / 2 % 8, so that the operand reads of 16 rows lie in different banks.
typedef __attribute__((address_space(3))) void lds_void;
template <int RT>
__global__ void __launch_bounds__(256) lora_shrink_tiled_kernel(LoraArgs p, int splits,
                                                                int shares) {
    constexpr int kA = RT > 1 ? RT / 2 : 1;               // copies of A a wavefront and step
    constexpr int kLoads = 2 + kA;
    constexpr int kXBytes = 8192, kStep = kXBytes + 4096 * kA;
    // distinct objects: the compiler tells copies into one from reads of another
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[kStep];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[kStep];
    __shared__ __attribute__((aligned(1024))) uint8_t buf2[kStep];
    __shared__ __attribute__((aligned(1024))) uint8_t buf3[kStep];
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) & 3;
    const int64_t tile = tile_of(p, blockIdx.x);
    if (tile < 0) return;
    const int64_t m0 = tile * 64;
    const int split = blockIdx.y % splits, rank0 = blockIdx.y / splits * (16 * RT);
    const int share = blockIdx.z;
    const int64_t Rp = (p.R + 15) / 16 * 16;
    const int steps = (int)((p.K + 63) / 64);
    const int s0 = (int)((int64_t)steps * split / splits);
    const int s1 = (int)((int64_t)steps * (split + 1) / splits);
    const int64_t left = p.M - m0 < 64 ? p.M - m0 : 64;
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(p.x + m0 * p.ldx, (uint32_t)(((left - 1) * p.ldx + p.K) * 2));
    const uint32_t row_bytes = (uint32_t)(p.K * 2);
    // a copy's lane: row lane / 8 of its eight rows 8 n .., the piece that belongs
    // at place lane % 8 of it
    auto piece = [&](int n) { return 16u * (uint32_t)((lane % 8) ^ (4 * (n % 2) + lane / 16)); };

    each_adapter(p, m0, 64, share, shares, [&](int g, uint64_t same) {
        const __amdgpu_buffer_rsrc_t ar =
            make_rsrc(p.a + (int64_t)g * p.R * p.K, (uint32_t)(p.R * p.K * 2));
        uint32_t xo[2], ao[kA];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 16 * wave + 8 * i + lane / 8;
            xo[i] = same >> row & 1 ? (uint32_t)(row * p.ldx * 2) + piece(i) : kOOB;
        }
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            const int n = 8 * (wave * kA + i) + lane / 8;
            ao[i] = n < 16 * RT && rank0 + n < p.R ? (uint32_t)(rank0 + n) * row_bytes +
                                                         piece(wave * kA + i)
                                                   : kOOB;
        }
        auto copy = [&](uint8_t *to, int s) {
            const uint32_t k = 128u * (uint32_t)s;
            // past the split, or past the row's end (K % 64 != 0): zeros
            auto past = [&](int n) { return s < s1 && k + piece(n) < row_bytes ? 0u : kOOB; };
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    xr, (lds_void *)(to + (2 * wave + i) * 1024), 16,
                    (int)(((xo[i] & ~kOOB) + k) | (xo[i] & kOOB) | past(i)), 0, 0, kNT);
#pragma unroll
            for (int i = 0; i < kA; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ar, (lds_void *)(to + kXBytes + (wave * kA + i) * 1024), 16,
                    (int)(((ao[i] & ~kOOB) + k) | (ao[i] & kOOB) | past(wave * kA + i)), 0, 0,
                    0);
        };
        v4f acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
        // At a step's start every wavefront has waited for its own copies of the
        // step (those of the next two may be out); behind the barrier all of
        // them are there, and the buffer of the step before is free.
        auto step = [&](const uint8_t *cur, uint8_t *ahead, int s) {
            __builtin_amdgcn_s_waitcnt(vmcnt_only(2 * kLoads));
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            copy(ahead, s + 3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = 16 * ((4 * h + j) ^ (r / 2));
                const v4u x = *reinterpret_cast<const v4u *>(cur + (16 * wave + r) * 128 + at);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const v4u a = *reinterpret_cast<const v4u *>(cur + kXBytes +
                                                                 (16 * t + r) * 128 + at);
                    acc[t] = mfma_bf16(as_bf16x8(a), as_bf16x8(x), acc[t]);
                }
            }
        };
        __syncthreads();                                  // the last adapter's buffers are free
        copy(buf0, s0);
        copy(buf1, s0 + 1);
        copy(buf2, s0 + 2);
        // whole rounds of four steps: those past s1 multiply zeros
        for (int s = s0; s < s1; s += 4) {
            step(buf0, buf3, s);
            step(buf1, buf0, s + 1);
            step(buf2, buf1, s + 2);
            step(buf3, buf2, s + 3);
        }
        // no copy (of zeros, behind the last step) stays under way
        __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
        // element i of lane (j, r): rank 4 j + i, row r of each 16 x 16 tile
        const int row = 16 * wave + r;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int rank = rank0 + 16 * t + 4 * j;
            if ((same >> row & 1) && rank < Rp)
                *reinterpret_cast<v4f *>(p.ws + ((int64_t)split * p.M + m0 + row) * Rp + rank) =
                    acc[t];
        }
    });
}

// NC: chunks of 32 ranks whose columns of B are loaded together.  STAGED: B's
// rows of the workgroup's columns go through LDS, in whole lines and once for
// both row groups; the operand-shaped loads (64 bytes of 16 rows, 8 R apart)
// cost 20 of 47 us at R = 64, N = 4096, M = 4096.  The tile's rows are shared out
// to RG groups of wavefronts, 16 MW rows each, and a workgroup covers 128 columns
// for every wavefront of a group.
template <int MT, int NC, bool STAGED>
__global__ void __launch_bounds__(64 * expand_waves(MT)) lora_expand_kernel(LoraArgs p, int splits,
                                                                            int shares) {
    constexpr int kExpandWaves = expand_waves(MT);
    constexpr int MW = MT < 2 ? MT : 2, RG = MT / MW, CG = kExpandWaves / RG;
    // v of the tile's rows: [chunks of 32 ranks][roundings, remainders][16 MT rows]
    // [4 pieces of 8 ranks], piece x of a row standing at x ^ (row / 4) % 4 so that
    // the 16 rows of one read lie in different banks
    constexpr int kV = STAGED ? NC * 2 * 16 * MT * 32 : 8;
    __shared__ __attribute__((aligned(16))) uint16_t vstatic[kV];
    extern __shared__ __attribute__((aligned(16))) uint16_t vdynamic[];
    uint16_t *const vs = STAGED ? vstatic : vdynamic;
    // B's rows of the workgroup's columns as they lie in memory, in 16-byte
    // pieces: piece q stands at q ^ (q >> s) % 16, 2^s <= R, which puts the 16 rows
    // of one read, R pieces apart, into different banks
    constexpr int kStaged = 128 * CG * 32 * NC * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t wlds[STAGED ? kStaged : 16];
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int rows0 = wave / CG * (16 * MW);              // this wavefront's first row in the tile
    // the tile is the fast grid axis: a tile's column groups run on one XCD, whose
    // L2 then holds its partial sums
    const int64_t tile = MT == 4 ? tile_of(p, blockIdx.x) : blockIdx.x;
    if (tile < 0) return;
    const int64_t m0 = tile * (16 * MT);
    const int64_t n0 = (int64_t)blockIdx.y * (128 * CG) + 128 * (wave % CG);
    const int share = blockIdx.z;
    const int Rp = (int)((p.R + 15) / 16 * 16), chunks = (Rp + 31) / 32;
    const int spread = p.R < 16 ? 4 : 31 - __builtin_clz((unsigned)p.R);
    const int64_t left = p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT;
    const __amdgpu_buffer_rsrc_t br =
        make_rsrc(p.base + m0 * p.ldb, (uint32_t)(((left - 1) * p.ldb + p.N) * 2));
    const __amdgpu_buffer_rsrc_t yr =
        make_rsrc(p.y + m0 * p.ldy, (uint32_t)(((left - 1) * p.ldy + p.N) * 2));
    // The products take v as the A and the adapter's rows as the B operand, column
    // 8 r + t of product t: element e of a lane is row 4 j + e, and its eight
    // products are eight neighbouring columns, so 16 lanes load and store 256
    // bytes of a row.  Byte offset of that piece of row 16 i + 4 j + e:
    auto place = [&](int i, int e, int64_t ld, uint64_t rows) {
        const int row = rows0 + 16 * i + 4 * j + e;
        const int64_t n = n0 + 8 * r;
        return (rows >> row & 1) && n < p.N ? (uint32_t)((row * ld + n) * 2) : kOOB;
    };

    // v of the rows in `rows`, zeros for the others
    auto stage = [&](uint64_t rows) {
        for (int n = threadIdx.x; n < 16 * MT * chunks * 8; n += 64 * kExpandWaves) {
            const int row = n / (chunks * 8), rank = n % (chunks * 8) * 4;
            v4f s = {0.f, 0.f, 0.f, 0.f};
            float scale = 1.0f;
            // (ranks from R on: zeros, not the products of A's missing rows, which an
            // infinite x turns into NaN)
            if ((rows >> row & 1) && rank < p.R) {
                if (p.scales) scale = p.scales[p.ids[m0 + row]];
                const float *at = p.ws + (m0 + row) * Rp + rank;
#pragma unroll 4
                for (int q = 0; q < splits; ++q)
                    s += *reinterpret_cast<const v4f *>(at + (int64_t)q * p.M * Rp);
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = s[i] * scale;
                hi[i] = __float_as_uint(v) >> 16;
                // (an infinity has no remainder: inf - inf would be NaN)
                lo[i] = (hi[i] & 0x7F80u) == 0x7F80u ? 0u : bf16_bits(v - bf16_to_f32(hi[i]));
            }
            uint16_t *to = vs + ((rank / 32) * 32 * MT + row) * 32 +
                           8 * ((rank % 32 / 8) ^ (row / 4 % 4)) + rank % 8;
            *reinterpret_cast<v2u *>(to) = v2u{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
            *reinterpret_cast<v2u *>(to + 16 * MT * 32) =
                v2u{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        }
    };

    // STAGED: v of the whole tile is staged with its first adapter; a product of
    // another adapter's row is not stored
    bool staged = false;
    const uint64_t all = each_adapter(p, m0, 16 * MT, share, shares, [&](int g, uint64_t same) {
        const __amdgpu_buffer_rsrc_t wr =
            make_rsrc(p.b + (int64_t)g * p.N * p.R, (uint32_t)(p.N * p.R * 2));
        auto load_w = [&](v4u (&w)[NC][8], int c0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int64_t n = n0 + 8 * r + t;
                    const int rank = 32 * (c0 + c) + 8 * j;
                    w[c][t] = load16(wr, n < p.N && rank < p.R ? (uint32_t)((n * p.R + rank) * 2)
                                                               : kOOB);
                }
        };
        auto read_w = [&](v4u (&w)[8], int c) {
            const int rank = 32 * c + 8 * j;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int q = ((128 * (wave % CG) + 8 * r + t) * (int)p.R + rank) / 8;
                w[t] = v4u{0u, 0u, 0u, 0u};
                if (rank < p.R)
                    w[t] = *reinterpret_cast<const v4u *>(wlds + 16 * (q ^ (q >> spread & 15)));
            }
        };
        // B's and the projection's loads go out ahead of the staging of v
        v4u w[NC][8], b[MW][4];
        __syncthreads();                                  // the last adapter's B and v are used up
        if constexpr (STAGED) {
            const uint32_t first = (uint32_t)(blockIdx.y * (128 * CG) * p.R * 2);
            for (int i = wave; 1024 * i < 128 * CG * p.R * 2; i += kExpandWaves) {
                const int at = 64 * i + lane;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    wr, (lds_void *)(wlds + 1024 * i), 16,
                    (int)(first + 16u * (uint32_t)(at ^ (at >> spread & 15))), 0, 0, 0);
            }
        } else {
            load_w(w, 0);
        }
#pragma unroll
        for (int i = 0; i < MW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) b[i][e] = load16<kNT>(br, place(i, e, p.ldb, same));
        if constexpr (STAGED) {
            if (!staged) {
                int id = -1;
                if (lane < left) id = p.ids[m0 + lane];
                stage(__ballot(id >= 0 && id < (int)p.L));
            }
            staged = true;
            __builtin_amdgcn_s_waitcnt(vmcnt_only(0));    // the copies have landed
        } else {
            stage(same);
        }
        __syncthreads();
        v4f acc[8][MW];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < MW; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
        auto products = [&](const v4u (&wc)[8], int c) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                v4u v[MW];
#pragma unroll
                for (int i = 0; i < MW; ++i)
                    v[i] = *reinterpret_cast<const v4u *>(
                        vs + ((c * 2 + f) * 16 * MT + rows0 + 16 * i + r) * 32 + 8 * (j ^ (r / 4)));
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int i = 0; i < MW; ++i)
                        acc[t][i] = mfma_bf16(as_bf16x8(v[i]), as_bf16x8(wc[t]), acc[t][i]);
            }
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (STAGED) read_w(w[c], c);
            if (c < chunks) products(w[c], c);
        }
        for (int c0 = NC; !STAGED && c0 < chunks; c0 += NC) {        // ranks beyond 32 NC
            load_w(w, c0);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (c0 + c < chunks) products(w[c], c0 + c);
        }
#pragma unroll
        for (int i = 0; i < MW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v4u o;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t u = b[i][e][d];
                    o[d] = bf16_bits(__uint_as_float(u << 16) + acc[2 * d][i][e]) |
                           bf16_bits(__uint_as_float(u & 0xFFFF0000u) + acc[2 * d + 1][i][e]) << 16;
                }
                __builtin_amdgcn_raw_buffer_store_b128(o, yr, (int)place(i, e, p.ldy, same), 0, 0);
            }
    });
    // rows without an adapter keep the projection
    if (share != 0 || (p.y == p.base && p.ldy == p.ldb)) return;
    const uint64_t none = ~all & (left < 64 ? (1ull << left) - 1 : ~0ull);
    if (!none) return;
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b128(load16(br, place(i, e, p.ldb, none)), yr,
                                                   (int)place(i, e, p.ldy, none), 0, 0);
}

template <int MT, int RT>
static void shrink(const LoraArgs &a, int splits, hipStream_t st) {
    const int64_t tiles = lora_tiles(a.M, MT), chunks = (a.R + 16 * RT - 1) / (16 * RT);
    const int shares = lora_shares(a.M, MT, tiles * splits * chunks, 1024);
    const dim3 grid((unsigned)grid_tiles(a.M, MT), (unsigned)(splits * chunks), (unsigned)shares);
    if constexpr (MT == 4)
        hipLaunchKernelGGL(lora_shrink_tiled_kernel<RT>, grid, dim3(256), 0, st, a, splits, shares);
    else
        hipLaunchKernelGGL(lora_shrink_kernel<RT>, grid, dim3(64 * kShrinkWaves), 0, st, a, splits,
                           shares);
}

template <int MT, int NC, bool STAGED>
static void expand(const LoraArgs &a, int splits, hipStream_t st) {
    constexpr int waves = expand_waves(MT), cols = 128 * (MT == 4 ? waves / 2 : waves);
    const int64_t tiles = lora_tiles(a.M, MT), groups = (a.N + cols - 1) / cols;
    // the staged form's LDS leaves two places a compute unit: none for idle ones
    const int shares = lora_shares(a.M, MT, tiles * groups, STAGED ? 512 : 1024);
    const unsigned lds = STAGED ? 0u : (unsigned)(16 * MT * ((a.R + 31) / 32) * 128);
    hipLaunchKernelGGL((lora_expand_kernel<MT, NC, STAGED>),
                       dim3((unsigned)grid_tiles(a.M, MT), (unsigned)groups, (unsigned)shares),
                       dim3(64 * waves), lds, st, a, splits, shares);
}

template <int MT>
static hipError_t launch_mt(const LoraArgs &a, hipStream_t st) {
    const int splits = (int)lora_splits(a.M, a.K, a.invariant);
    if (a.R <= 16) shrink<MT, 1>(a, splits, st);
    else if (a.R <= 32) shrink<MT, 2>(a, splits, st);
    else shrink<MT, 4>(a, splits, st);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (a.R <= 32) expand<MT, 1, MT == 4>(a, splits, st);
    else if (a.R <= 64) expand<MT, 2, MT == 4>(a, splits, st);
    else expand<MT, 2, false>(a, splits, st);
    return hipGetLastError();
}

hipError_t launch_lora(const LoraArgs &a, hipStream_t st) {
    return lora_mt(a.M, a.invariant) == 4 ? launch_mt<4>(a, st) : launch_mt<1>(a, st);
}

}  // namespace mx
