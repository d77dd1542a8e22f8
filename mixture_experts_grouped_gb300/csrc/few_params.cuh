// What the few-token layer's kernels take.
#pragma once

#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

struct FewParams {
    const uint16_t* x;
    const float* logits;   // or NULL: ids / weights are inputs
    int32_t* ids;
    float* weights;
    int T, k, H, I, E, renorm;
    MoeWeight gu, down;
    uint16_t* h;           // [slots, I]
    uint16_t* out;
    int32_t* err;
};

}  // namespace moe
