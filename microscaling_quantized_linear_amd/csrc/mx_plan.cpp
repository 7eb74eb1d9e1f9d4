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

// The plan of the GEMV that quantizes inside, with an epilogue: four tiles a workgroup
// instead of two, for seven steps a wavefront (K 7168 alone: the steps divide evenly),
// where that takes fewer rounds of 256
// workgroups by more than a third, a round of four tiles being about half as long again.
// Measured, us at four / two (K 7168): one round against two, M 16, N 9216 15.2 / 19.2,
// N 14336 18.5 / 20.8, N 16384 20.4 / 21.6, M 32, N 7168 14.6 / 19.9; two against four,
// M 64, N 7168 27.8 / 37.5; three against five, M 40, N 12288 42.5 / 48.4.  Not where it
// is one against one, N 8192 14.8 / 12.0, or two against three, N 20480 31.6 / 29.1 (M
// 48, N 7168: 26.4 / 28.4).  Eight steps a wavefront lose (N 16384, K 8192: 29.6 / 27.6).
GemvW8Plan gemv_w8_fused_epi_plan(int64_t N, int64_t M, const GemvW8Plan &given) {
    GemvW8Plan pl = given;
    const int64_t T = N / 16, MB = (M + 15) / 16;
    auto rounds = [&](int64_t g) { return (T / g * MB + 255) / 256; };
    if (pl.spw == 7 && pl.g == 2 && T % 4 == 0 && 3 * rounds(4) < 2 * rounds(2)) pl.g = 4;
    return pl;
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
