// mx_lanes.h -- exchanges between the lanes of a wavefront that need no LDS: DPP
// within rows of 16 lanes, v_permlane16_swap and v_permlane32_swap across them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace mx {

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kRotate8 = 0x128;

// f over groups of LPT neighbouring lanes; every lane gets the result.  Lanes 16 apart
// meet first, then 32, 8, and those of eight neighbours.
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
    if (LPT >= 16) v = f(v, dpp<kRotate8>(v));
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
// how many of the LPT <= 16 neighbouring lanes hold a larger value
template <int LPT>
__device__ inline int lanes_ahead(uint32_t v) {
    int n = 0;
    auto count = [&](uint32_t u) { n += u > v ? 1 : 0; };
    if constexpr (LPT == 16) {
        // DPP row_ror 1 .. 15
        count(dpp<0x121>(v)); count(dpp<0x122>(v)); count(dpp<0x123>(v)); count(dpp<0x124>(v));
        count(dpp<0x125>(v)); count(dpp<0x126>(v)); count(dpp<0x127>(v)); count(dpp<0x128>(v));
        count(dpp<0x129>(v)); count(dpp<0x12A>(v)); count(dpp<0x12B>(v)); count(dpp<0x12C>(v));
        count(dpp<0x12D>(v)); count(dpp<0x12E>(v)); count(dpp<0x12F>(v));
    } else if constexpr (LPT == 8) {
        // the other seven: quad permutations of this quad and of the mirrored one
        const uint32_t m = dpp<kHalfMirror>(v);
        count(dpp<0xB1>(v)); count(dpp<0x4E>(v)); count(dpp<0x1B>(v)); count(m);
        count(dpp<0xB1>(m)); count(dpp<0x4E>(m)); count(dpp<0x1B>(m));
    }
    return n;
}
// the sum over a group's lanes up to and with this one
template <int LPT>
__device__ inline int lanes_prefix(int v) {
    const int i = (int)threadIdx.x % LPT;
    // DPP row_shr 1, 2, 4, 8: zeros come in at a row's start
    auto shr = [&](int u, auto step, uint32_t got) { return u + (i >= decltype(step)::value ? (int)got : 0); };
    v = shr(v, std::integral_constant<int, 1>{}, dpp<0x111>((uint32_t)v));
    v = shr(v, std::integral_constant<int, 2>{}, dpp<0x112>((uint32_t)v));
    v = shr(v, std::integral_constant<int, 4>{}, dpp<0x114>((uint32_t)v));
    if (LPT >= 16) v = shr(v, std::integral_constant<int, 8>{}, dpp<0x118>((uint32_t)v));
    if (LPT >= 32) {
        const int before = __shfl(v, ((int)threadIdx.x % 64 & ~31) + 15);
        v += i % 32 >= 16 ? before : 0;
    }
    if (LPT == 64) {
        const int before = __shfl(v, 31);
        v += i >= 32 ? before : 0;
    }
    return v;
}
// the same of 64-bit values as over_lanes32
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
        v = f(v, whole(dpp<kRotate8>(lo), dpp<kRotate8>(hi)));
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
