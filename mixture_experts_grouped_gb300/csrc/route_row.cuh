// Top-k softmax routing of one row by one warp, shared by the routing kernel,
// the fused router kernel and the few-token layer, so all take the same
// decisions in the same arithmetic.
#pragma once

#include <math.h>

#include "common.cuh"

namespace moe {

constexpr int kPerLane = MOE_MAX_EXPERTS / 32;  // 8

__device__ __forceinline__ bool better(float va, int ia, float vb, int ib) {
    return va > vb || (va == vb && ia < ib);
}

// Top-k softmax of one row whose logits sit in registers: lane l holds
// v[j] = logit of expert l + 32 j (E <= 256). Writes the row's top_k ids and
// weights (lanes < top_k).
__device__ __forceinline__ void route_row(const float (&v)[kPerLane], int lane, int E, int k, int renorm,
                                          int32_t* __restrict__ ids_row, float* __restrict__ w_row) {
    uint32_t taken = 0;  // bit j: element lane + 32 j already selected (or absent)
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
        if (lane + 32 * j >= E) taken |= 1u << j;

    int sel_i[MOE_MAX_TOPK];
    float sel_v[MOE_MAX_TOPK];
#pragma unroll
    for (int r = 0; r < MOE_MAX_TOPK; ++r) {
        sel_i[r] = 0;
        sel_v[r] = 0.0f;
        if (r >= k) continue;
        float bv = 0.0f;
        int bi = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            const int i = lane + 32 * j;
            if (!(taken >> j & 1u) && (bi == 0x7fffffff || better(v[j], i, bv, bi))) {
                bv = v[j];
                bi = i;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
            if (oi != 0x7fffffff && (bi == 0x7fffffff || better(ov, oi, bv, bi))) {
                bv = ov;
                bi = oi;
            }
        }
        if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
        sel_i[r] = bi;
        sel_v[r] = bv;
    }

    const float m = sel_v[0];
    // lane r < k holds the exponential of its selected expert: the fp64 exp is
    // evaluated once per selected expert, in parallel across the lanes
    float sv = 0.0f;
    int si = 0;
#pragma unroll
    for (int q = 0; q < MOE_MAX_TOPK; ++q)
        if (q == lane) {
            sv = sel_v[q];
            si = sel_i[q];
        }
    const float e_mine = (lane < k) ? __double2float_rn(exp(static_cast<double>(__fsub_rn(sv, m)))) : 0.0f;
    float denom;
    if (renorm) {
        denom = 0.0f;  // e_0 + e_1 + ... in rank order
#pragma unroll
        for (int r = 0; r < MOE_MAX_TOPK; ++r) {
            const float er = __shfl_sync(0xffffffffu, e_mine, r);
            if (r < k) denom = __fadd_rn(denom, er);
        }
    } else {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            if (lane + 32 * j < E)
                part = __fadd_rn(part, __double2float_rn(exp(static_cast<double>(__fsub_rn(v[j], m)))));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) part = __fadd_rn(part, __shfl_xor_sync(0xffffffffu, part, off));
        denom = part;
    }
    if (lane < k) {
        ids_row[lane] = si;
        w_row[lane] = __fdiv_rn(e_mine, denom);
    }
}

}  // namespace moe
