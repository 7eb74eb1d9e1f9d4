// mx_plan.cpp -- host-only launch plans of the W8A8 decode GEMV (kept out of
// the kernel sources so the host logic builds alone, e.g. with sanitizers).
#include "mx_kernels.h"

namespace mx {

// (K % 128 == 0: the even kernels step through whole 2 KB chunks, S per tile)
bool gemv_w8_even(int64_t N, int64_t K, const GemvW8Plan &pl) {
    const int64_t S = K / 128, T = N / 16;
    return K % 128 == 0 && pl.ok && pl.nw == 8 && S == 8 * (int64_t)pl.spw && T % pl.g == 0 &&
           pl.g * pl.spw <= 16;
}

// Weight rows of a tile of the prefill GEMM with an epilogue: the fewest, 64 or 128, at
// which every tile of 256 tokens has a compute unit of its own; from more than 256
// tiles of 128 rows on, those of mx_linear (224 or 256).  A tile's time is its
// products, a step of 128 K at 0.92 us for 256 rows, and its epilogue, one wavefront a
// SIMD: with idle compute units both shrink with the tile.  Measured, us at 256 / 128 /
// 64 rows (K 1568, GELU and residual): M 512, N 2048 28.8 / 16.4 / 10.6; M 1001, N 4096
// 30.3 / 17.8 / 13.2; M 2048, N 4096 33.6 / 23.6 / 23.7; M 3000, N 4096 36.8 / 37.0 /
// 34.5; M 4096, N 7168 66.9 / 76.6 / 71.7 (K 7168: 170 / 197 / 213).
int gemm_epi_tile_n(int64_t M, int64_t N) {
    const int64_t mt = (M + 255) / 256;
    for (int bn : {64, 128})
        if ((N + bn - 1) / bn * mt <= 256) return bn;
    return gemm_tile_n(N);
}

// Launch plan for T tiles, S steps and MB 16-token grid rows: tiles per
// workgroup G in {4, 2, 1} (the largest that still gives about one
// workgroup per compute unit, measured best on MI355X), up to eight
// wavefronts per workgroup, each with at most SPW in {1, 2, 4, 7, 8} steps.
// ok = false when S needs more than 64 steps' worth of registers.  nw_force
// and g_force (0 = none) override the choice, for tuning sweeps.
GemvW8Plan plan_gemv_w8(int64_t T, int64_t S, int64_t MB, int nw_force, int g_force) {
    GemvW8Plan pl{};
    int nw = S >= 8 ? 8 : (int)S;
    if (nw_force >= 1 && nw_force <= 8) nw = nw_force;
    const int64_t per = (S + nw - 1) / nw;
    pl.nw = nw;
    pl.spw = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : per == 7 ? 7 : 8;
    pl.ok = per <= 8;
    pl.g = 1;
    for (int g : {4, 2}) {
        if (g * pl.spw > 16) continue;                   // register budget
        if ((T + g - 1) / g * MB >= 224) {
            pl.g = g;
            break;
        }
    }
    if ((g_force == 1 || g_force == 2 || g_force == 4) && g_force * pl.spw <= 16) pl.g = g_force;
    return pl;
}

}  // namespace mx
