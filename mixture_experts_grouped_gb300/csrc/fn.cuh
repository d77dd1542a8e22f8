// The activation functions of the dense product and their derivatives, in f32.
#pragma once

#include "quant.cuh"

namespace moe {

// 1 / (1 + exp(-z)) by the hardware's 2^x and reciprocal, a few ulp; 0 below
// z = -87.3 (the reciprocal's flush), 1 at +inf.
__device__ __forceinline__ float sigmoid_fast(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504088896341f));  // log2(e)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// g s and its slope, of s = sigmoid_fast(g). A gate stored in 16 bits may have overflowed: an infinite one has its limits,
// 0 and 0 at -inf, inf and 1 at +inf (g s alone and g (1 - s) would be NaN). A NaN is in s, and stays.
__device__ __forceinline__ float silu_part(float g, float s) { return fmaxf(g, -3.402823466e38f) * s; }
__device__ __forceinline__ float silu_slope(float g, float s) {
    const float c = fminf(fmaxf(g, -100.0f), 100.0f);  // beyond, s (1 - s) is 0
    return s * fmaf(c, 1.0f - s, 1.0f);
}

// sqrt(2 / pi) (z + 0.044715 z^3), doubled: (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)),
// which keeps its relative accuracy where 1 + tanh v cancels
__device__ __forceinline__ float gelu_tanh_arg2(float z) {
    return z * fmaf(0.0713548162726f, z * z, 1.59576912160573f);  // 2 sqrt(2 / pi) (0.044715, 1)
}

// The normal distribution at z, from e = exp(-z^2 / 2). Of x = |z| it is t P(t) exp(-x^2 / 2) on the negative side,
// t = 1 / (1 + 0.36 x), P of degree 6: the minimax fit of Phi(-x) exp(x^2 / 2) / t over 0 <= x <= 14, relative, by
// Remez' exchange in 64 bits (8.7e-7; the scale in t is the one whose fit is best). So the far tail keeps its relative
// accuracy: 1.3e-6 to z = -3, 7e-6 at z = -13, where the exponent's rounding is the larger part. A third of the
// instructions of the library's erfc, which bounded the gradient below.
__device__ __forceinline__ float normal_cdf(float z, float e) {
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.36f, fabsf(z), 1.0f)));
    float q = fmaf(t, 0.0470560603f, -0.179763898f);
    q = fmaf(t, q, 0.180952936f);
    q = fmaf(t, q, 0.0265500285f);
    q = fmaf(t, q, 0.139719024f);
    q = fmaf(t, q, 0.141772494f);
    q = fmaf(t, q, 0.143713042f) * t * e;
    return z < 0.0f ? q : 1.0f - q;
}
__device__ __forceinline__ float exp_minus_half_square(float z) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -0.72134752044448170f));  // log2(e) / 2
    return e;
}

// f(z). Functions are chosen per launch, so FN is uniform and the branches cost nothing.
__device__ __forceinline__ float fn_value(int fn, float z) {
    switch (fn) {
        case MOE_FN_RELU: return z < 0.0f ? 0.0f : z;  // (NaN stays)
        case MOE_FN_GELU: return z * normal_cdf(z, exp_minus_half_square(z));
        case MOE_FN_GELU_TANH: return z * sigmoid_fast(gelu_tanh_arg2(z));
        case MOE_FN_SILU: return z * sigmoid_fast(z);
        default: return z;
    }
}

// f of eight values: one branch for all, and as little code as that takes
__device__ __forceinline__ void fn_values(int fn, float (&f)[8]) {
    switch (fn) {
        case MOE_FN_RELU:
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fn_value(MOE_FN_RELU, f[j]);
            break;
        case MOE_FN_GELU:
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fn_value(MOE_FN_GELU, f[j]);
            break;
        case MOE_FN_GELU_TANH:
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fn_value(MOE_FN_GELU_TANH, f[j]);
            break;
        case MOE_FN_SILU:
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fn_value(MOE_FN_SILU, f[j]);
            break;
        default: break;
    }
}

// f'(z), at an infinity its limit: a z that is finite in f32 may be stored as one in 16 bits. NaN stays.
__device__ __forceinline__ float fn_slope(int fn, float z) {
    switch (fn) {
        case MOE_FN_RELU: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
        case MOE_FN_GELU: {
            const float c = fminf(fmaxf(z, -40.0f), 40.0f);  // beyond, the density is 0 and must not meet an infinity
            const float e = exp_minus_half_square(z);
            return fmaf(c * 0.398942280401432678f, e, normal_cdf(z, e));
        }
        case MOE_FN_GELU_TANH: {
            const float c = fminf(fmaxf(z, -20.0f), 20.0f);  // beyond, s (1 - s) is 0
            const float s = sigmoid_fast(gelu_tanh_arg2(z));
            return fmaf(c * s * (1.0f - s), fmaf(0.2140644488178f, c * c, 1.59576912160573f), s);
        }
        case MOE_FN_SILU: return silu_slope(z, sigmoid_fast(z));
        default: return 1.0f;
    }
}

}  // namespace moe
