// mx_route.hip -- the order of routed (token, choice) pairs by expert, and the
// weighted sum of a token's expert outputs.
//
// Sort.  Pair i (token i / topk) goes to expert ids[i]; an id outside [0, E)
// counts as expert E, whose pairs come last and have no place.  The order is
// the stable one: place(i) = offsets[ids[i]] + the number of earlier pairs of
// the same expert.  A counting sort: a histogram per part of the pairs, then
// every part's pairs placed behind those of the earlier parts.  Within a part
// each wavefront takes consecutive pairs, 64 at a time; a lane's rank among the
// lanes of its expert comes from one ballot per bit of the expert number, so
// the result never depends on timing.
//   bounds: at decode sizes the launch and two passes over a few kilobytes
//   (latency); at prefill sizes 12 bytes a pair.
// Up to kSmall pairs one workgroup does it all; more pairs are cut into parts
// of at least kSmall pairs, one workgroup each, with the parts' histograms in
// the workspace between two launches.
#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int64_t kSmall = 2048;           // pairs of one part, at least
constexpr int64_t kMaxParts = 256;

static int64_t sort_parts(int64_t pairs) {
    const int64_t n = (pairs + kSmall - 1) / kSmall;
    return n < kMaxParts ? n : kMaxParts;
}
// whole groups of 64 pairs per wavefront
static int64_t part_pairs(int64_t pairs) {
    const int64_t n = sort_parts(pairs), unit = 64 * kSortWaves;
    return ((pairs + n - 1) / n + unit - 1) / unit * unit;
}

// a part's histogram: E + 1 counts, padded with zeros to whole 16 bytes
__host__ __device__ inline int hist_row(int E) { return (E + 4) / 4 * 4; }

int64_t moe_sort_ws_bytes(int64_t E, int64_t pairs) {
    const int64_t n = sort_parts(pairs);
    return n > 1 ? n * hist_row((int)E) * 4 : 0;
}

__device__ inline int expert_of(const int32_t *ids, int64_t i, int64_t end, int E) {
    if (i >= end) return -1;                              // no pair
    const int32_t id = ids[i];
    return id >= 0 && id < E ? id : E;
}

// Histogram of each wavefront's pairs in cnt[wave][0 .. E]: wavefront w of
// part [first, end) takes the `per` pairs from first + w * per on.  The experts
// of its first kKept groups of 64 pairs stay in `kept`.
constexpr int kKept = 4;
__device__ inline void count_part(const int32_t *ids, int64_t first, int64_t end, int64_t per,
                                  int E, int *cnt, int bins, int (&kept)[kKept]) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t at = first + wave * per + lane;
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        kept[i] = 64 * i < per ? expert_of(ids, at + 64 * i, end, E) : -1;
    for (int b = threadIdx.x; b < kSortWaves * bins; b += kSortThreads) cnt[b] = 0;
    __syncthreads();
    // whole numbers: the order of the additions does not show
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (kept[i] >= 0) atomicAdd(&cnt[wave * bins + kept[i]], 1);
    for (int64_t i = 64 * kKept; i < per; i += 64) {
        const int e = expert_of(ids, at + i, end, E);
        if (e >= 0) atomicAdd(&cnt[wave * bins + e], 1);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(
    const int32_t *__restrict__ ids, int64_t pairs, int64_t part, int E,
    int32_t *__restrict__ hist) {
    extern __shared__ int cnt[];
    const int bins = E + 1;
    const int64_t first = blockIdx.x * part, end = first + part < pairs ? first + part : pairs;
    int kept[kKept];
    count_part(ids, first, end, part / kSortWaves, E, cnt, bins, kept);
    for (int b = threadIdx.x; b < hist_row(E); b += kSortThreads) {
        int n = 0;
        for (int w = 0; b < bins && w < kSortWaves; ++w) n += cnt[w * bins + b];
        hist[(int64_t)blockIdx.x * hist_row(E) + b] = n;
    }
}

// Places the pairs of part blockIdx.x.  hist: the parts' histograms, or null
// when this is the only part.
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(
    const int32_t *__restrict__ ids, int64_t pairs, int64_t part, int E, int topk, int bits,
    const int32_t *__restrict__ hist, int32_t *__restrict__ offsets, int32_t *__restrict__ rows,
    int32_t *__restrict__ pos) {
    extern __shared__ int cnt[];                          // [waves][bins], total[bins], base[bins]
    __shared__ int wsum[kSortWaves];
    const int bins = E + 1;
    int *total = cnt + kSortWaves * bins, *base = total + bins;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t first = blockIdx.x * part, end = first + part < pairs ? first + part : pairs;
    const int64_t per = part / kSortWaves;
    int kept[kKept];
    // total[b]: every part's pairs of expert b; base[b]: those in earlier parts.
    // A thread reads four experts' counts at once and, where the experts are few,
    // several threads share their parts.
    for (int b = threadIdx.x; b < 2 * bins; b += kSortThreads) total[b] = 0;
    count_part(ids, first, end, per, E, cnt, bins, kept);
    if (hist) {
        const int quads = hist_row(E) / 4, parts = (int)gridDim.x;
        const int teams = kSortThreads / quads > 0 ? kSortThreads / quads : 1;
        for (int i = threadIdx.x; i < teams * quads; i += kSortThreads) {
            const int b = i % quads * 4;
            v4i before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
#pragma unroll 8
            for (int q = i / quads; q < parts; q += teams) {
                const v4i n = *reinterpret_cast<const v4i *>(hist + (int64_t)q * quads * 4 + b);
                if (q < (int)blockIdx.x) before += n;
                all += n;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b + k < bins) {
                    atomicAdd(&total[b + k], all[k]);
                    atomicAdd(&base[b + k], before[k]);
                }
        }
        __syncthreads();
    }
    // cnt[w][b]: the pairs of expert b ahead of wavefront w's
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        int before = base[b];
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = cnt[w * bins + b];
            cnt[w * bins + b] = before;
            before += n;
        }
        if (!hist) total[b] = before;
    }
    __syncthreads();
    // exclusive sums of total over the experts, 512 bins at a time
    int carry = 0;
    for (int base = 0; base < bins; base += kSortThreads) {
        const int b = base + threadIdx.x;
        const int n = b < bins ? total[b] : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(inc, o);
            inc += lane >= o ? v : 0;
        }
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int up = carry, sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            up += w < wave ? wsum[w] : 0;
            sum += wsum[w];
        }
        if (b < bins) total[b] = up + inc - n;
        carry += sum;
        __syncthreads();
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < bins; b += kSortThreads) offsets[b] = total[b];
    // the pairs, 64 of a wavefront at a time and in order.  LDS operations of a
    // wavefront complete in order; the compiler is told to keep them so.
    auto wave_order = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
    };
    int *mine = cnt + wave * bins;
    auto put = [&](int e, int64_t pair) {
        uint64_t same = __ballot(e >= 0);
        for (int bit = 0; bit < bits; ++bit) {
            const uint64_t on = __ballot(e >> bit & 1);
            same &= e >> bit & 1 ? on : ~on;
        }
        if (e >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1ull));
            const int at = mine[e] + rank;
            const int place = total[e] + at;
            rows[place] = e < E ? (int32_t)((uint32_t)pair / (uint32_t)topk) : -1;
            pos[pair] = e < E ? place : -1;
            // the last lane of the expert moves its count on, once every lane
            // of the wavefront has read it
            wave_order();
            if (rank == __popcll(same) - 1) mine[e] = at + 1;
        }
        wave_order();
    };
    const int64_t at = first + wave * per + lane;
#pragma unroll
    for (int i = 0; i < kKept; ++i) put(kept[i], at + 64 * i);
    for (int64_t i = 64 * kKept; i < per; i += 64) put(expert_of(ids, at + i, end, E), at + i);
}

hipError_t launch_moe_sort(int64_t E, int64_t pairs, int64_t topk, const int32_t *ids,
                           int32_t *offsets, int32_t *rows, int32_t *pos, void *ws,
                           hipStream_t st) {
    const int64_t n = sort_parts(pairs), part = part_pairs(pairs);
    const unsigned bins = (unsigned)E + 1, lds = kSortWaves * bins * 4;
    int bits = 1;
    while ((int64_t(1) << bits) <= E) ++bits;             // experts 0 .. E
    int32_t *hist = n > 1 ? static_cast<int32_t *>(ws) : nullptr;
    if (n > 1) {
        hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)n), dim3(kSortThreads), lds, st, ids,
                           pairs, part, (int)E, hist);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(moe_place_kernel, dim3((unsigned)n), dim3(kSortThreads), lds + 2 * bins * 4,
                       st, ids, pairs, part, (int)E, (int)topk, bits, hist, offsets, rows, pos);
    return hipGetLastError();
}

// Combine.  y[t][n] = sum_k w[t][k] ys[pos[t][k]][n], in k order in fp32 and
// rounded once; a choice whose place is outside [0, M) adds nothing (its row
// is not read).  One workgroup a token and 2048 columns, eight columns a
// thread; the choices' rows are read four at a time (eight: the same), past the
// caches, as nothing reads them again (T = 4096, topk 8, N = 7168, 505 MB: 104 ->
// 90 us, 5.6 TB/s).  HBM-bound: topk + 1 rows of 2 N bytes a token.
__global__ void __launch_bounds__(256) moe_gather_sum_kernel(
    int topk, int64_t N, int64_t M, const uint16_t *__restrict__ ys, int64_t ldys,
    const int32_t *__restrict__ pos, const float *__restrict__ wts, uint16_t *__restrict__ y,
    int64_t ldy) {
    const int64_t t = blockIdx.x;
    const int64_t n = 2048 * (int64_t)blockIdx.y + 8 * threadIdx.x;
    if (n >= N) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < topk; k0 += 4) {
        v4u v[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t at = k0 + u < topk ? pos[t * topk + k0 + u] : -1;
            const bool ok = at >= 0 && at < M;
            w[u] = ok ? wts[t * topk + k0 + u] : 0.0f;
            v[u] = v4u{0u, 0u, 0u, 0u};
            if (ok)
                v[u] = __builtin_nontemporal_load(
                    reinterpret_cast<const v4u *>(ys + at * ldys + n));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                acc[2 * d] = __builtin_fmaf(w[u], __uint_as_float(v[u][d] << 16), acc[2 * d]);
                acc[2 * d + 1] = __builtin_fmaf(w[u], __uint_as_float(v[u][d] & 0xFFFF0000u),
                                                acc[2 * d + 1]);
            }
    }
    v4u o;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = bf16_bits(acc[2 * d]) | bf16_bits(acc[2 * d + 1]) << 16;
    *reinterpret_cast<v4u *>(y + t * ldy + n) = o;
}

hipError_t launch_moe_gather_sum(int64_t T, int64_t topk, int64_t N, int64_t M, const uint16_t *ys,
                                 int64_t ldys, const int32_t *pos, const float *wts, uint16_t *y,
                                 int64_t ldy, hipStream_t st) {
    hipLaunchKernelGGL(moe_gather_sum_kernel, dim3((unsigned)T, (unsigned)((N + 2047) / 2048)),
                       dim3(256), 0, st, (int)topk, N, M, ys, ldys, pos, wts, y, ldy);
    return hipGetLastError();
}

}  // namespace mx
