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

// the tensor-core form (block_fp8_tc.cu)
int launch_block_fp8_tc(const BfParams& p, int act, int sms, int32_t* err, cudaStream_t st, const char* who);

}  // namespace moe
