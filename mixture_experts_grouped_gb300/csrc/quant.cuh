// E4M3 quantisation with one f32 scale per 128 columns, shared by the
// operators that write it.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kQuantGroup = 128;                    // columns per scale
constexpr int kQuantLanes = kQuantGroup / 8;        // lanes of 8 columns per group: half a warp
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;        // 2^-126: the scale of an all-zero group, and its reciprocal is finite

// max |v| as the bits of a non-negative float: unsigned order is the order of
// the magnitudes, and a NaN's bits lie above infinity's, so it wins.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}
// the same over the 16 lanes of a half warp (every lane of the warp calls it)
__device__ __forceinline__ uint32_t amax_half_warp(uint32_t m) {
#pragma unroll
    for (int off = kQuantLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}
// scale = max(amax / 448, 2^-126); a NaN amax stays NaN
__device__ __forceinline__ float group_scale(uint32_t bits) {
    const float s = __fdiv_rn(__uint_as_float(bits), kE4m3Max);
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
