// What the two forms of the block-scaled E4M3 product take.
#pragma once

#include "quant.cuh"

namespace moe {

struct BfParams {
    const uint8_t* a;
    const float* sa;
    const uint8_t* w;
    const float* sb;
    const uint16_t* addend;
    uint16_t* out;
    int M, N, K, kb;  // kb: scales per row
};

// A block's sum v is scaled by two f32 values a and b as v * f, f = a * b rounded
// once: one product more per block, none per element. f may overflow, or lose
// bits below the normal range, where v * a * b does neither (|v| is 0 or between
// 2^-18 and 2^25). Then v takes the scales one after the other, the larger
// first: if f overflows, the smaller is above 1, so v times the larger overflows
// only where the result does; if f is subnormal, the larger is below 2^23 (the
// smaller is 2^-149 at least), and v times it is normal where the result is.
// Returns the factor for v before f (1 as a rule): v * a * b = (v * before) * f.
__device__ __forceinline__ float scale_before(float& f, float a, float b) {
    if (((__float_as_uint(f) >> 23 & 255u) - 1u) < 254u || a == 0.0f || b == 0.0f) return 1.0f;
    const bool swap = fabsf(a) < fabsf(b);
    f = swap ? a : b;
    return swap ? b : a;
}
// A quick look at f: true for 2^-63 <= |f| < 2^65 (the exponent's two upper bits
// differ), which needs nothing before it.
__device__ __forceinline__ bool scale_ordinary(float f) {
    const uint32_t u = __float_as_uint(f);
    return (u ^ u << 1) >> 30 & 1u;
}

// the tensor-core form (block_fp8_tc.cu)
int launch_block_fp8_tc(const BfParams& p, int act, int sms, int32_t* err, cudaStream_t st, const char* who);

}  // namespace moe
