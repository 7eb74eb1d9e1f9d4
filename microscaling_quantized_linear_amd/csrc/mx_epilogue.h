// mx_epilogue.h -- what the dense products do behind their sums when a call has
// an epilogue (mx_linear_epilogue): bias, activation, gate, residual, one rounding.
//
//   z = sum + bias,  h[n] = f(z[n])  or, gated,  f(z[2 n]) * z[2 n + 1],
//   y = bf16(h + residual), all of it in fp32.
// The kernels are compiled a second time with it (EPI), so those of calls
// without one stay as they are.
#pragma once

#include <cfloat>
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

// The activations by what they cost: none, relu and relu2 are comparisons and a
// product; silu and tanh-gelu are z times a logistic function, of z and of an odd
// cubic (0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))), each in a form of its own: a cubic
// with a zero coefficient is NaN where z is infinite; erf-gelu has its own.
// (KIND_NONE: the prefill kernel's form for none.)
enum { KIND_SIMPLE = 0, KIND_SILU = 1, KIND_TANH = 2, KIND_ERF = 3, KIND_NONE = 4 };
__host__ __device__ inline int fn_kind(int fn) {
    return fn == FN_GELU        ? KIND_ERF
           : fn == FN_GELU_TANH ? KIND_TANH
           : fn == FN_SILU      ? KIND_SILU
                                : KIND_SIMPLE;
}

struct FnCoef {
    bool relu, square;
};
__device__ inline FnCoef fn_coef(int fn) {
    FnCoef c;
    c.relu = fn == FN_RELU || fn == FN_RELU2;
    c.square = fn == FN_RELU2;
    return c;
}

// f(z).  KIND_SILU, KIND_TANH: z / (1 + 2^t), t of the other sign than z, both parts
// times 2^-8.  v_rcp_f32 gives 0 for a divisor above 2^126, which is 2^t alone at z =
// -87.3 (silu) where z / 2^t is 2^-119 yet; scaled, the divisor gets there at t = 134
// only, where the quotient is below 2^-126.  v_exp_f32 and v_rcp_f32 are within a last
// place; with the exponent's roundings the value is within 4e-6 (silu) and 1.1e-5 of
// itself at the left end, within 3e-7 right of zero (7e-6 where z 2^-8 is below
// 2^-126): far below the bf16 rounding that follows.  Infinite z give the limits:
// 2^-inf is 0 and z itself remains, and on the left the largest number stands for z,
// whose quotient is 0 (NaN stays in t).
// KIND_ERF: z Phi(z) with Phi(-t) = exp(-t^2 / 2) p(1 / (1 + 0.42 t / sqrt 2)), p of
// degree 6 fitted to 0.5 erfcx in relative error (1.8e-6; with the roundings, the
// exponent's two among them, 4e-6 for t <= 8 and 1e-5 at t = 13, where |z Phi(z)| is
// 2^-126), so the negative tail keeps its relative precision too.
template <int KIND>
__device__ inline float fn_value(float z, const FnCoef &c) {
    if constexpr (KIND == KIND_SILU || KIND == KIND_TANH) {
        constexpr double kLog2e = 1.4426950408889634, kTanh = -1.5957691216057308 * kLog2e;
        // tanh-gelu: -2 sqrt(2 / pi) (z + 0.044715 z^3) log2 e
        const float a = KIND == KIND_SILU
                            ? (float)-kLog2e
                            : __builtin_fmaf(z * (float)(0.044715 * kTanh), z, (float)kTanh);
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, a, -8.0f));       // 2^(t - 8)
        return __builtin_fmaxf(z * 0x1p-8f, -FLT_MAX) * __builtin_amdgcn_rcpf(0x1p-8f + e);
    } else if constexpr (KIND == KIND_ERF) {
        const float t = __builtin_fminf(__builtin_fabsf(z), 32.0f);
        const float u = __builtin_amdgcn_rcpf(__builtin_fmaf(t, 0.42f * 0.70710678f, 1.0f));
        float q = -8.709728153423472e-2f;
        q = __builtin_fmaf(q, u, 2.5824102861334264e-1f);
        q = __builtin_fmaf(q, u, -6.904218537505563e-2f);
        q = __builtin_fmaf(q, u, 1.7540824306243566e-1f);
        q = __builtin_fmaf(q, u, 1.0198490649281536e-1f);
        q = __builtin_fmaf(q, u, 1.2061959005405326e-1f);
        q = __builtin_fmaf(q, u, -1.1386800506109441e-4f);
        const float e = __builtin_amdgcn_exp2f(t * t * -0.72134752044448170f);
        return __builtin_fmaf(-t, q * e, z < 0.0f ? 0.0f : z);
    } else if constexpr (KIND == KIND_NONE) {
        return z;
    } else {
        const float r = c.relu && z < 0.0f ? 0.0f : z;
        return c.square ? r * r : r;
    }
}

// the same of n values, by a function known at run time only (uniform branches)
template <int n>
__device__ inline void fn_any(int fn, float (&v)[n], const FnCoef &c) {
    auto each = [&](auto kind) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = fn_value<decltype(kind)::value>(v[i], c);
    };
    const int kind = fn_kind(fn);
    if (kind == KIND_SIMPLE) each(std::integral_constant<int, KIND_SIMPLE>{});
    else if (kind == KIND_SILU) each(std::integral_constant<int, KIND_SILU>{});
    else if (kind == KIND_TANH) each(std::integral_constant<int, KIND_TANH>{});
    else each(std::integral_constant<int, KIND_ERF>{});
}

// The decode kernels' epilogue: a lane holds the sums of weight rows n0 .. n0 + 3
// (n0 % 4 == 0) for one token row.
struct EpiLane {
    uint32_t bias[4];
    v2u res;          // bf16 of four columns, or of two (dword 0) when gated
};
__device__ inline EpiLane epi_load(const EpiArgs &f, const uint16_t *bias, int64_t n0, int64_t row) {
    EpiLane e;
    if (bias)
        for (int i = 0; i < 4; ++i) e.bias[i] = bias[n0 + i];
    e.res = v2u{0u, 0u};
    if (f.res) {
        if (f.gated)
            e.res[0] = *reinterpret_cast<const uint32_t *>(f.res + row * f.ldr + n0 / 2);
        else
            e.res = *reinterpret_cast<const v2u *>(f.res + row * f.ldr + n0);
    }
    return e;
}
__device__ inline void epi_store(const EpiArgs &f, const uint16_t *bias, const EpiLane &e, v4f a,
                                 int64_t n0, int64_t row, uint16_t *y, int64_t ldy) {
    const FnCoef c = fn_coef(f.fn);
    float v[4] = {a[0], a[1], a[2], a[3]};
    if (bias)
        for (int i = 0; i < 4; ++i) v[i] += bf16_to_f32(e.bias[i]);
    if (f.gated) {
        float h[2] = {v[0], v[2]};
        fn_any(f.fn, h, c);
        for (int i = 0; i < 2; ++i) {
            h[i] *= v[2 * i + 1];
            if (f.res) h[i] += i ? __uint_as_float(e.res[0] & 0xFFFF0000u) : bf16_to_f32(e.res[0]);
        }
        *reinterpret_cast<uint32_t *>(y + row * ldy + n0 / 2) = bf16_bits(h[0]) | bf16_bits(h[1]) << 16;
        return;
    }
    fn_any(f.fn, v, c);
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = e.res[i / 2];
        if (f.res) v[i] += i % 2 ? __uint_as_float(r & 0xFFFF0000u) : bf16_to_f32(r);
    }
    *reinterpret_cast<v2u *>(y + row * ldy + n0) =
        v2u{bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
}

}  // namespace mx
