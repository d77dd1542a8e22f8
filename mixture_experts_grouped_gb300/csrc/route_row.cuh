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

// The weights of a row whose selection is known: lane r < k holds the r-th
// expert si and its logit sv, m is the largest logit. Writes the row's ids and
// weights (lanes < top_k).
__device__ __forceinline__ void finish_row(const float (&v)[kPerLane], int lane, int E, int k, int renorm, float m,
                                           float sv, int si, int32_t* __restrict__ ids_row,
                                           float* __restrict__ w_row) {
    // lane r < k holds the exponential of its selected expert: the fp64 exp is
    // evaluated once per selected expert, in parallel across the lanes
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

    // lane r takes the r-th selection
    float sv = 0.0f;
    int si = 0;
#pragma unroll
    for (int q = 0; q < MOE_MAX_TOPK; ++q)
        if (q == lane) {
            sv = sel_v[q];
            si = sel_i[q];
        }
    finish_row(v, lane, E, k, renorm, sel_v[0], sv, si, ids_row, w_row);
}

// The selection of route_row by integer reductions, of up to ROWS rows at once
// (their reductions overlap), for E <= 32 PER: lane r < k gets the r-th expert
// of row q in si[q] and its logit in sv[q]. Each round takes the largest
// remaining logit as an order-preserving integer with one warp reduction, and
// the lowest index that holds it with a second. Returns the rows that hold a
// NaN, bit by bit: nothing is selected for them (route_row's comparisons are
// not an order then). (route_row itself took about 8 us of a one-token layer
// when every CTA ran it: its 16 unrolled rounds of shuffles, and the fp64
// exponential, which runs on few units per SM.)
template <int PER, int ROWS>
__device__ __forceinline__ uint32_t select_rows_n(const float* const (&lrow)[ROWS], int rows, int lane, int E, int k,
                                                  float (&sv)[ROWS], int (&si)[ROWS]) {
    uint32_t key[ROWS][PER], nan = 0;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const bool in = q < rows && lane + 32 * j < E;
            const float v = in ? __ldg(lrow[q] + lane + 32 * j) : 0.0f;
            bad |= v != v;
            const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));  // -0 counts as 0
            // 0: absent or taken
            key[q][j] = in ? b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u) : 0u;
        }
        nan |= static_cast<uint32_t>(bad) << q;
        sv[q] = 0.0f;
        si[q] = 0;
    }
    nan = __reduce_or_sync(0xffffffffu, nan);
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            if (q > 0 && q >= rows) break;
            uint32_t bk = key[q][0];
#pragma unroll
            for (int j = 1; j < PER; ++j) bk = max(bk, key[q][j]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
            uint32_t mine = ~0u;
#pragma unroll
            for (int j = PER - 1; j >= 0; --j)
                if (key[q][j] == top) mine = lane + 32 * j;
            const uint32_t at = __reduce_min_sync(0xffffffffu, mine);
            if (lane == r) {
                si[q] = static_cast<int>(at);
                sv[q] = __uint_as_float((top & 0x80000000u) ? top & 0x7fffffffu : ~top);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 32 * j == at) key[q][j] = 0u;
        }
    }
    return nan;
}
template <int ROWS>
__device__ __forceinline__ uint32_t select_rows(const float* const (&lrow)[ROWS], int rows, int lane, int E, int k,
                                                float (&sv)[ROWS], int (&si)[ROWS]) {
    return E <= 128 ? select_rows_n<4, ROWS>(lrow, rows, lane, E, k, sv, si)
                    : select_rows_n<kPerLane, ROWS>(lrow, rows, lane, E, k, sv, si);
}

}  // namespace moe
