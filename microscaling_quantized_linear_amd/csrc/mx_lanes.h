// mx_lanes.h -- exchanges between the lanes of a wavefront that need no LDS: DPP
// within rows of 16 lanes, v_permlane16_swap and v_permlane32_swap across them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// f over groups of LPT neighbouring lanes; every lane gets the result.  The distant
// lanes meet first.
template <int LPT, class F>
__device__ inline uint32_t over_lanes32(uint32_t v, F f) {
    if (LPT >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    if (LPT == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    if (LPT >= 16) v = f(v, dpp<kMirror>(v));
    v = f(v, dpp<kHalfMirror>(v));
    v = f(v, dpp<kSwap2>(v));
    return f(v, dpp<kSwap1>(v));
}
template <int LPT>
__device__ inline float lanes_sum(float v) {
    return __uint_as_float(over_lanes32<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int LPT>
__device__ inline float lanes_max(float v) {
    return __uint_as_float(over_lanes32<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
// the same of 64-bit values
template <int LPT, class F>
__device__ inline double over_lanes64(double v, F f) {
    auto halves = [](double d, uint32_t &lo, uint32_t &hi) {
        const uint64_t u = __builtin_bit_cast(uint64_t, d);
        lo = (uint32_t)u;
        hi = (uint32_t)(u >> 32);
    };
    auto whole = [](uint32_t lo, uint32_t hi) {
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    };
    uint32_t lo, hi;
    if (LPT >= 32) {
        halves(v, lo, hi);
        const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        v = f(whole(a[0], b[0]), whole(a[1], b[1]));
    }
    if (LPT == 64) {
        halves(v, lo, hi);
        const auto a = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        v = f(whole(a[0], b[0]), whole(a[1], b[1]));
    }
    if (LPT >= 16) {
        halves(v, lo, hi);
        v = f(v, whole(dpp<kMirror>(lo), dpp<kMirror>(hi)));
    }
    halves(v, lo, hi);
    v = f(v, whole(dpp<kHalfMirror>(lo), dpp<kHalfMirror>(hi)));
    halves(v, lo, hi);
    v = f(v, whole(dpp<kSwap2>(lo), dpp<kSwap2>(hi)));
    halves(v, lo, hi);
    return f(v, whole(dpp<kSwap1>(lo), dpp<kSwap1>(hi)));
}

// LDS operations of a wavefront complete in order; the compiler is told to keep them so
__device__ inline void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace mx
