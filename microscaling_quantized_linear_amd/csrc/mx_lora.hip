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
//   expand  v as the sum of two bf16 numbers (its rounding and the rounding's
//           remainder, 16 significant bits): of the 32 values of K of one
//           matrix-core product the first 16 hold the roundings and the last
//           16 the remainders, both against the same 16 columns of B, so the
//           second part costs no further product and v loses nothing that the
//           bf16 result would show.  The residual of the projection is added in
//           fp32 and y rounded once.
// Bounds: at decode the adapters' bytes, 2 R (N + K) each, and two launches'
// latency; at prefill x, base and y, 2 K + 4 N bytes a row.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4, kExpandCols = 64 * kExpandWaves;

// rows of a tile, in units of 16
static int lora_mt(int64_t M) { return M >= 512 ? 4 : 1; }
static int64_t lora_tiles(int64_t M) {
    const int64_t t = 16 * lora_mt(M);
    return (M + t - 1) / t;
}
// K splits of the shrink: 2048 values (256 a wavefront) each where the rows
// are few, fewer splits once the tiles alone give about two workgroups a
// compute unit
int64_t lora_splits(int64_t M, int64_t K) {
    const int64_t most = (K + 2047) / 2048, tiles = lora_tiles(M);
    const int64_t want = (512 + tiles - 1) / tiles;
    return want < most ? want : most;
}
// workgroups that share a tile's adapters
static int lora_shares(int64_t M, int64_t groups) {
    const int64_t most = 16 * lora_mt(M), want = (512 + groups - 1) / groups;
    const int64_t g = want < most ? want : most;
    return (int)(g < M ? g : M);
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

template <int MT, int RT>
__global__ void __launch_bounds__(64 * kShrinkWaves) lora_shrink_kernel(LoraArgs p, int splits,
                                                                        int shares) {
    __shared__ v4f red[kShrinkWaves][MT][64];
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t m0 = (int64_t)blockIdx.x * (16 * MT);
    const int split = blockIdx.y % splits, rank0 = blockIdx.y / splits * (16 * RT);
    const int share = blockIdx.z;
    const int64_t Rp = (p.R + 15) / 16 * 16;
    // this wavefront's units of 32 values of K
    const int units = (int)(p.K / 32), parts = splits * kShrinkWaves;
    const int part = split * kShrinkWaves + wave;
    const int u0 = (int)((int64_t)units * part / parts);
    const int u1 = (int)((int64_t)units * (part + 1) / parts);
    const int64_t left = p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT;
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(p.x + m0 * p.ldx, (uint32_t)(((left - 1) * p.ldx + p.K) * 2));
    const uint32_t row_bytes = (uint32_t)(p.K * 2);

    each_adapter(p, m0, 16 * MT, share, shares, [&](int g, uint64_t same) {
        const __amdgpu_buffer_rsrc_t ar =
            make_rsrc(p.a + (int64_t)g * p.R * p.K, (uint32_t)(p.R * p.K * 2));
        uint32_t xo[MT], ao[RT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
            xo[t] = same >> (16 * t + r) & 1 ? (uint32_t)((16 * t + r) * p.ldx * 2 + 16 * j) : kOOB;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int rank = rank0 + 16 * t + r;
            ao[t] = rank < p.R ? (uint32_t)rank * row_bytes + 16u * j : kOOB;
        }
        v4f acc[RT][MT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
        constexpr int P = RT * MT >= 8 ? 2 : 4;           // units loaded together
        for (int u = u0; u < u1; u += P) {
            v4u a[P][RT], x[P][MT];
#pragma unroll
            for (int q = 0; q < P; ++q) {
                // a unit past the wavefront's range reads zeros
                const uint32_t k = u + q < u1 ? 64u * (uint32_t)(u + q) : kOOB;
#pragma unroll
                for (int t = 0; t < RT; ++t) a[q][t] = load16(ar, (ao[t] + (k & ~kOOB)) | (ao[t] & kOOB) | (k & kOOB));
#pragma unroll
                for (int t = 0; t < MT; ++t) x[q][t] = load16(xr, (xo[t] + (k & ~kOOB)) | (xo[t] & kOOB) | (k & kOOB));
            }
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[t][i] = mfma_bf16(as_bf16x8(a[q][t]), as_bf16x8(x[q][i]), acc[t][i]);
        }
        // element i of lane (j, r): rank 4 j + i, token r of each 16 x 16 tile
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[t][i];
            __syncthreads();
            for (int n = threadIdx.x; n < MT * 64; n += 64 * kShrinkWaves) {
                const int i = n / 64, l = n % 64;
                v4f s = red[0][i][l];
#pragma unroll
                for (int w = 1; w < kShrinkWaves; ++w) s += red[w][i][l];
                const int row = 16 * i + l % 16, rank = rank0 + 16 * t + 4 * (l / 16);
                if ((same >> row & 1) && rank < Rp)
                    *reinterpret_cast<v4f *>(p.ws + ((int64_t)split * p.M + m0 + row) * Rp + rank) = s;
            }
            __syncthreads();
        }
    });
}

template <int MT>
__global__ void __launch_bounds__(64 * kExpandWaves) lora_expand_kernel(LoraArgs p, int splits,
                                                                        int shares) {
    // v of the tile's rows: [16 MT rows][Rp / 16 chunks][16 roundings, 16 remainders]
    extern __shared__ __attribute__((aligned(16))) uint16_t vs[];
    const int lane = threadIdx.x % 64, r = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int64_t n0 = (int64_t)blockIdx.x * kExpandCols + 64 * wave;
    const int share = blockIdx.z;
    const int Rp = (int)((p.R + 15) / 16 * 16);
    const int64_t left = p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT;
    const __amdgpu_buffer_rsrc_t br =
        make_rsrc(p.base + m0 * p.ldb, (uint32_t)(((left - 1) * p.ldb + p.N) * 2));
    const __amdgpu_buffer_rsrc_t yr =
        make_rsrc(p.y + m0 * p.ldy, (uint32_t)(((left - 1) * p.ldy + p.N) * 2));
    const int64_t nl = n0 + 16 * j;                       // this lane's 16 columns

    const uint64_t all = each_adapter(p, m0, 16 * MT, share, shares, [&](int g, uint64_t same) {
        const float scale = p.scales ? p.scales[g] : 1.0f;
        __syncthreads();                                  // the last adapter's v is used up
        for (int n = threadIdx.x; n < 16 * MT * Rp / 4; n += 64 * kExpandWaves) {
            const int row = n / (Rp / 4), rank = n % (Rp / 4) * 4;
            v4f s = {0.f, 0.f, 0.f, 0.f};
            if (same >> row & 1)
                for (int q = 0; q < splits; ++q)
                    s += *reinterpret_cast<const v4f *>(p.ws + ((int64_t)q * p.M + m0 + row) * Rp +
                                                        rank);
            uint16_t *to = vs + (row * (Rp / 16) + rank / 16) * 32 + rank % 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = s[i] * scale;
                const uint32_t hi = bf16_bits(v);
                to[i] = (uint16_t)hi;
                to[16 + i] = (uint16_t)bf16_bits(v - bf16_to_f32(hi));
            }
        }
        __syncthreads();
        const __amdgpu_buffer_rsrc_t wr =
            make_rsrc(p.b + (int64_t)g * p.N * p.R, (uint32_t)(p.N * p.R * 2));
        v4f acc[4][MT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < Rp / 16; ++c) {
            v4u w[4], v[MT];
            // row 4 a + b of product t is column 16 a + 4 t + b, so that a
            // lane's four products give 16 neighbouring columns
            const int rank = 16 * c + 8 * (j % 2);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t n = n0 + 16 * (r / 4) + 4 * t + r % 4;
                w[t] = load16(wr, n < p.N && rank < p.R ? (uint32_t)((n * p.R + rank) * 2) : kOOB);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                v[i] = *reinterpret_cast<const v4u *>(vs + ((16 * i + r) * (Rp / 16) + c) * 32 + 8 * j);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[t][i] = mfma_bf16(as_bf16x8(w[t]), as_bf16x8(v[i]), acc[t][i]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = 16 * i + r;
            const bool mine = (same >> row & 1) && nl < p.N;
            const uint32_t bo = mine ? (uint32_t)((row * p.ldb + nl) * 2) : kOOB;
            const uint32_t yo = mine ? (uint32_t)((row * p.ldy + nl) * 2) : kOOB;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u b = load16(br, bo + 16u * h);
                v4u o;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int t = 2 * h + d / 2, e = 2 * (d % 2);
                    o[d] = bf16_bits(__uint_as_float(b[d] << 16) + acc[t][i][e]) |
                           bf16_bits(__uint_as_float(b[d] & 0xFFFF0000u) + acc[t][i][e + 1]) << 16;
                }
                __builtin_amdgcn_raw_buffer_store_b128(o, yr, (int)(yo + 16u * h), 0, 0);
            }
        }
    });
    // rows without an adapter keep the projection
    if (share != 0 || (p.y == p.base && p.ldy == p.ldb)) return;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = 16 * i + r;
        const bool copy = !(all >> row & 1) && m0 + row < p.M && nl < p.N;
        const uint32_t bo = copy ? (uint32_t)((row * p.ldb + nl) * 2) : kOOB;
        const uint32_t yo = copy ? (uint32_t)((row * p.ldy + nl) * 2) : kOOB;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            __builtin_amdgcn_raw_buffer_store_b128(load16(br, bo + 16u * h), yr,
                                                   (int)(yo + 16u * h), 0, 0);
    }
}

template <int MT, int RT>
static void shrink(const LoraArgs &a, int splits, hipStream_t st) {
    const int64_t tiles = lora_tiles(a.M), chunks = (a.R + 16 * RT - 1) / (16 * RT);
    const int shares = lora_shares(a.M, tiles * splits * chunks);
    hipLaunchKernelGGL((lora_shrink_kernel<MT, RT>),
                       dim3((unsigned)tiles, (unsigned)(splits * chunks), (unsigned)shares),
                       dim3(64 * kShrinkWaves), 0, st, a, splits, shares);
}

template <int MT>
static hipError_t launch_mt(const LoraArgs &a, hipStream_t st) {
    const int splits = (int)lora_splits(a.M, a.K);
    if (a.R <= 16) shrink<MT, 1>(a, splits, st);
    else if (a.R <= 32) shrink<MT, 2>(a, splits, st);
    else shrink<MT, 4>(a, splits, st);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t tiles = lora_tiles(a.M), cols = (a.N + kExpandCols - 1) / kExpandCols;
    const int shares = lora_shares(a.M, tiles * cols);
    const unsigned lds = (unsigned)(16 * MT * ((a.R + 15) / 16) * 64);
    hipLaunchKernelGGL((lora_expand_kernel<MT>),
                       dim3((unsigned)cols, (unsigned)tiles, (unsigned)shares),
                       dim3(64 * kExpandWaves), lds, st, a, splits, shares);
    return hipGetLastError();
}

hipError_t launch_lora(const LoraArgs &a, hipStream_t st) {
    return lora_mt(a.M) == 4 ? launch_mt<4>(a, st) : launch_mt<1>(a, st);
}

}  // namespace mx
