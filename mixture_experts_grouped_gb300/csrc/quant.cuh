// E4M3 quantisation with one f32 scale per 128 columns, shared by the
// operators that write it.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kQuantGroup = 128;                    // columns per scale
constexpr int kQuantLanes = kQuantGroup / 8;        // lanes of 8 columns per group: half a warp
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;        // 2^-126: the scale of an all-zero group, and its reciprocal is finite

// the larger, or NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
    return m;
}
// the same over the 16 lanes of a half warp; `mask` names the lanes that call it
__device__ __forceinline__ float amax_half_warp(float m, uint32_t mask) {
#pragma unroll
    for (int off = kQuantLanes / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(mask, m, off));
    return m;
}
// scale = max(amax / 448, 2^-126); a NaN amax stays NaN
__device__ __forceinline__ float group_scale(float amax) {
    const float s = __fdiv_rn(amax, kE4m3Max);
    return s < kMinScale ? kMinScale : s;
}
// four codes, the first in the lowest byte; rounds to nearest even, saturates at 448
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// Codes of eight values under scale s. The quotient is taken as v * (1 / s):
// within 1.5 ulp of v / s, so a code differs from the exact quotient's only
// where that lies within 2^-22 of a rounding boundary.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float s) {
    const float r = __frcp_rn(s);
    uint2 q;
    q.x = e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
    q.y = e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
    return q;
}

// silu(g) * u = g / (1 + exp(-g)) * u by the hardware's 2^x and reciprocal, with
// subnormals flushed: where exp(-g) would be subnormal, 1 + it is 1 either way,
// and below g = -87.3, where the reciprocal would be (|silu(g)| < 1.1e-36),
// the product is a zero.
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504088896341f));  // log2(e)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

// eight 16-bit activations <-> f32
template <int ACT> __device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Act<ACT>::unpack2(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <int ACT> __device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(Act<ACT>::pack2(v[0], v[1]), Act<ACT>::pack2(v[2], v[3]), Act<ACT>::pack2(v[4], v[5]),
                      Act<ACT>::pack2(v[6], v[7]));
}

}  // namespace moe
