// The whole expert layer for at most 32 tokens, in two kernels.
//
//     h[t, j, :] = act( silu(x[t] . Wg_e) * (x[t] . Wu_e) ),  e = ids[t, j]
//     out[t]     = act( sum_j w[t, j] * (h[t, j] . Wd_e) )
//
// With few tokens the layer is bound by the touched experts' weight bytes, and
// at one or two tokens as much by latency, so nothing stands between the
// routing and the weight stream: no sort, no gather, no padding, and no
// separate combine. Both kernels rebuild the same small plan in shared memory
// from the ids (routing the tokens themselves when given logits): a bit mask
// of tokens per expert (T <= 32 bits), the touched experts in ascending order
// and, per expert, its "slots" (distinct tokens, ascending) with their summed
// weights. Each CTA then takes an equal share of the weight rows:
//   gate/up  rows (touched expert, i), one share of consecutive rows per CTA,
//            8 gate and the 8 up rows of the same i to a product of 16 rows,
//            so one lane holds both sums of an h element. The contraction is
//            split over the CTA's warps and added through shared memory.
//   down     columns [n0, n1) of every touched expert, so the weighted sum
//            over the experts stays inside the CTA: each warp keeps its own
//            f32 sums per token in shared memory and adds an expert's products,
//            times the weight, when it leaves that expert; the warps' sums are
//            added in warp order. No atomics: results do not depend on timing.
#pragma once

#include "few_params.cuh"
#include "route_row.cuh"
#include "stream.cuh"

namespace moe {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewRing = 8;  // units a warp has in flight
constexpr int kFewPairs = MOE_MAX_FEW_TOKENS * MOE_MAX_TOPK;

struct FewPlan {
    int n;                              // touched experts
    int te[MOE_MAX_EXPERTS];            // touched experts, ascending
    int start[MOE_MAX_EXPERTS + 1];     // first slot of each
    uint32_t mask[MOE_MAX_EXPERTS];     // by expert id: tokens routed to it
    int first[MOE_MAX_EXPERTS];         // by expert id: first slot
    int ids[kFewPairs];
    float pw[kFewPairs];
    float slot_w[kFewPairs];
    uint8_t slot_tok[kFewPairs];
    uint32_t scan[kFewWarps];
};

// Fills the plan. `publish`: this CTA writes the routing outputs and reports bad ids.
__device__ __forceinline__ void build_plan(FewPlan& s, const FewParams& p, bool publish) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.T * p.k;
    static_assert(kFewThreads >= MOE_MAX_EXPERTS, "one thread per expert");
    if (tid < MOE_MAX_EXPERTS) s.mask[tid] = 0;
    if (p.logits) {
        for (int t = warp; t < p.T; t += kFewWarps) {
            float v[kPerLane];
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                const int e = lane + 32 * j;
                v[j] = e < p.E ? __ldg(p.logits + t * p.E + e) : 0.0f;
            }
            route_row(v, lane, p.E, p.k, p.renorm, s.ids + t * p.k, s.pw + t * p.k);
        }
    } else {
        for (int i = tid; i < P; i += kFewThreads) {
            s.ids[i] = p.ids[i];
            s.pw[i] = p.weights[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < P; i += kFewThreads) {
        const int e = s.ids[i];
        if (e >= 0 && e < p.E) atomicOr(&s.mask[e], 1u << (i / p.k));
        else if (publish) set_err(p.err, MOE_DEV_ERR_EXPERT_ID);
        if (publish && p.logits) {
            p.ids[i] = e;
            p.weights[i] = s.pw[i];
        }
    }
    __syncthreads();
    // prefix sums over the experts: touched experts in the high half, slots in the low
    const uint32_t m = tid < MOE_MAX_EXPERTS ? s.mask[tid] : 0u;
    const uint32_t mine = (m ? 1u << 16 : 0u) + __popc(m);
    uint32_t inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) s.scan[warp] = inc;
    __syncthreads();
    uint32_t before = inc - mine;
    for (int w = 0; w < warp; ++w) before += s.scan[w];
    if (m) {
        const int i = before >> 16;
        s.te[i] = tid;
        s.start[i] = before & 0xffffu;
        s.first[tid] = before & 0xffffu;
    }
    if (tid == kFewThreads - 1) {
        const uint32_t all = before + mine;
        s.n = all >> 16;
        s.start[all >> 16] = all & 0xffffu;
    }
    __syncthreads();
    for (int i = tid; i < P; i += kFewThreads) {
        const int e = s.ids[i], t = i / p.k, end = (t + 1) * p.k;
        if (e < 0 || e >= p.E) continue;
        bool again = false;
        for (int j = t * p.k; j < i; ++j) again |= s.ids[j] == e;
        if (again) continue;
        float w = s.pw[i];
        for (int j = i + 1; j < end; ++j)
            if (s.ids[j] == e) w += s.pw[j];
        const int slot = s.first[e] + __popc(s.mask[e] & ((1u << t) - 1u));
        s.slot_tok[slot] = static_cast<uint8_t>(t);
        s.slot_w[slot] = w;
    }
    __syncthreads();
}

// ---- gate/up ----------------------------------------------------------------------

// Position of a warp in its CTA's rows: item (touched expert, up to 8 columns
// i) and contraction step.
struct GuCursor {
    int r, end;      // row = touched index * I + i
    int ti, i, cnt;  // the item
    int j;           // contraction step
    __device__ __forceinline__ void init(int r0, int r1, int I) {
        r = r0;
        end = r1;
        ti = r0 / I;
        i = r0 - ti * I;
        cnt = min(8, min(end - r, I - i));
        j = 0;
    }
    __device__ __forceinline__ bool done() const { return r >= end; }
    __device__ __forceinline__ void next(int nk, int I) {
        if (++j < nk) return;
        j = 0;
        r += cnt;
        i += cnt;
        if (i == I) {
            i = 0;
            ++ti;
        }
        cnt = min(8, min(end - r, I - i));
    }
};

template <int FMT, int ACT, int NT>
__global__ void __launch_bounds__(kFewThreads, 2) few_gate_up_kernel(const FewParams p) {
    using U = Unit<FMT, ACT>;
    extern __shared__ float4 few_smem[];
    float4* red = few_smem;  // [2][warps][NT][32]: the warps' sums of an item
    __shared__ FewPlan s;
    pdl_wait();
    pdl_launch_next();  // the down kernel's CTAs set up beside this kernel's and wait for its end
    build_plan(s, p, blockIdx.x == 0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int I = p.I, K = p.H;
    const int64_t rows = static_cast<int64_t>(s.n) * I;
    const int r0 = static_cast<int>(rows * blockIdx.x / gridDim.x);
    const int r1 = static_cast<int>(rows * (blockIdx.x + 1) / gridDim.x);
    if (r0 >= r1) return;
    const int nk = ((K + U::SPAN - 1) / U::SPAN + kFewWarps - 1) / kFewWarps;  // steps per warp and item

    U ring[kFewRing];
    GuCursor ld, cs;
    ld.init(r0, r1, I);
    cs.init(r0, r1, I);
    WBase wb = expert_base<FMT>(p.gu.w, p.gu.scales, p.gu.zeros, 2 * I, K, p.gu.group_size, s.te[ld.ti]);
    int lti = ld.ti;
    auto fetch = [&](U& u) {
        if (ld.done()) return;
        if (ld.ti != lti) {
            lti = ld.ti;
            wb = expert_base<FMT>(p.gu.w, p.gu.scales, p.gu.zeros, 2 * I, K, p.gu.group_size, s.te[lti]);
        }
        const int row = g < ld.cnt ? ld.i + g : -1;
        u.load(wb, row, row < 0 ? -1 : I + row, (ld.j * kFewWarps + warp) * U::SPAN, c);
        ld.next(nk, I);
    };
#pragma unroll
    for (int d = 0; d < kFewRing; ++d) fetch(ring[d]);

    float acc[NT][4];
    const uint16_t* xp[NT];
    int nt = 0, parity = 0;
    while (!cs.done()) {
#pragma unroll
        for (int d = 0; d < kFewRing; ++d) {
            if (cs.done()) break;
            const int s0 = s.start[cs.ti], ns = s.start[cs.ti + 1] - s0;
            if (cs.j == 0) {  // a new item
                nt = (ns + 7) / 8;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int q = 8 * t + g;
                    xp[t] = q < ns ? p.x + static_cast<size_t>(s.slot_tok[s0 + q]) * K : nullptr;
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                }
            }
            unit_mma<FMT, ACT, NT>(ring[d], xp, nt, (cs.j * kFewWarps + warp) * U::SPAN, K, c, acc);
            if (cs.j == nk - 1) {  // the item's contraction is complete: add the warps' sums
                const float f0 = U::ROW_SCALE ? ring[d].scale(0) : 1.0f, f1 = U::ROW_SCALE ? ring[d].scale(1) : 1.0f;
                float4* mine = red + (parity * kFewWarps + warp) * NT * 32;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < nt)
                        mine[t * 32 + lane] =
                            make_float4(f0 * acc[t][0], f0 * acc[t][1], f1 * acc[t][2], f1 * acc[t][3]);
                __syncthreads();
                // thread (slot, row): 8 rows per slot
                const int slot = tid >> 3, row = tid & 7;
                if (slot < ns && row < cs.cnt) {
                    const float* src = reinterpret_cast<const float*>(
                        red + (parity * kFewWarps * NT + (slot >> 3)) * 32 + row * 4 + ((slot & 7) >> 1));
                    float gs = 0.0f, us = 0.0f;
#pragma unroll
                    for (int w = 0; w < kFewWarps; ++w) {
                        gs += src[w * NT * 128 + (slot & 1)];
                        us += src[w * NT * 128 + 2 + (slot & 1)];
                    }
                    if (FMT == MOE_W_NVFP4) {
                        gs *= __ldg(p.gu.scale2 + s.te[cs.ti]);
                        us *= __ldg(p.gu.scale2 + p.E + s.te[cs.ti]);
                    }
                    const float v = __fdividef(gs, 1.0f + __expf(-gs)) * us;
                    reinterpret_cast<typename Act<ACT>::T*>(p.h)[static_cast<size_t>(s0 + slot) * I + cs.i + row] =
                        Act<ACT>::from_f(v);
                }
                parity ^= 1;  // the next item writes the other half; the one after, behind the next barrier
            }
            cs.next(nk, I);
            fetch(ring[d]);
        }
    }
}

// ---- down ---------------------------------------------------------------------------

// The end of a 16-column tile: adds the warps' sums in warp order, writes the
// columns and clears the sums for the next tile.
template <int ACT>
__device__ __noinline__ void few_tile_end(float* sums, uint16_t* out, int T, int H, int n0, int n1) {
    __syncthreads();
    for (int i = threadIdx.x; i < T * 16; i += kFewThreads) {
        const int tok = i >> 4, col = i & 15;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            float& part = sums[(w * T + tok) * 17 + col];
            v += part;
            part = 0.0f;
        }
        if (n0 + col < n1)
            reinterpret_cast<typename Act<ACT>::T*>(out)[static_cast<size_t>(tok) * H + n0 + col] =
                Act<ACT>::from_f(v);
    }
    __syncthreads();
}

template <int FMT, int ACT, int NT>
__global__ void __launch_bounds__(kFewThreads, 2) few_down_kernel(const FewParams p) {
    using U = Unit<FMT, ACT>;
    extern __shared__ float4 few_smem[];
    float* sums = reinterpret_cast<float*>(few_smem);  // [warps][T][17]: sums of 16 columns (and a pad)
    __shared__ FewPlan s;
    // reads only what was complete before the gate/up kernel started: logits, or ids and weights
    build_plan(s, p, false);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int K = p.I, n = s.n;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.H) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.H) * (blockIdx.x + 1) / gridDim.x);
    const int ntiles = (n1 - n0 + 15) / 16;
    const int nks = (K + U::SPAN - 1) / U::SPAN;
    float* mine = sums + warp * p.T * 17;
    for (int i = tid; i < kFewWarps * p.T * 17; i += kFewThreads) sums[i] = 0.0f;

    // A tile's units (touched expert, contraction step) are dealt to the warps
    // in turn from the tile's start; settle moves to the unit at or after a
    // position.
    auto settle = [&](int& tile, int& ti, int& ks) {
        while (ks >= nks && tile < ntiles) {
            ks -= nks;
            if (++ti >= n) {
                ti = 0;
                ks = warp;
                ++tile;
            }
        }
    };
    U ring[kFewRing];
    int ltile = n > 0 ? 0 : ntiles, lti = 0, lks = warp, lbase = -1;  // where the loads are
    WBase wb{};
    auto fetch = [&](U& u) {
        if (ltile >= ntiles) return;
        if (lti != lbase) {
            lbase = lti;
            wb = expert_base<FMT>(p.down.w, p.down.scales, p.down.zeros, p.H, K, p.down.group_size, s.te[lti]);
        }
        const int a = n0 + 16 * ltile + g;
        u.load(wb, a < n1 ? a : -1, a + 8 < n1 ? a + 8 : -1, lks * U::SPAN, c);
        lks += kFewWarps;
        settle(ltile, lti, lks);
    };
    settle(ltile, lti, lks);
#pragma unroll
    for (int d = 0; d < kFewRing; ++d) fetch(ring[d]);
    pdl_wait();       // h is complete
    __syncthreads();  // the sums are zero

    int ctile = n > 0 ? 0 : ntiles, cti = 0, cks = warp;  // where the products are
    settle(ctile, cti, cks);
    float acc[NT][4], f0 = 1.0f, f1 = 1.0f;
    const uint16_t* xp[NT];
    int nt = 0, at = -1;  // acc holds products of touched expert `at`
    auto leave_expert = [&]() {
        if (at < 0) return;
        const int s0 = s.start[at], ns = s.start[at + 1] - s0;
        const float s2 = FMT == MOE_W_NVFP4 ? __ldg(p.down.scale2 + s.te[at]) : 1.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int slot = 8 * t + 2 * c + q;
                if (slot < ns) {
                    float* dst = mine + s.slot_tok[s0 + slot] * 17 + g;
                    const float w = s.slot_w[s0 + slot] * s2;
                    dst[0] = fmaf(w, f0 * acc[t][q], dst[0]);
                    dst[8] = fmaf(w, f1 * acc[t][2 + q], dst[8]);
                }
            }
        }
        __syncwarp();  // another lane adds to the same token's sums for the next expert
        at = -1;
    };
    int tile = 0;
    while (tile < ntiles) {
#pragma unroll
        for (int d = 0; d < kFewRing; ++d) {
            if (tile < ctile) {  // no more units of this tile (and of any the warp has none of)
                leave_expert();
                for (; tile < ctile; ++tile)
                    few_tile_end<ACT>(sums, p.out, p.T, p.H, n0 + 16 * tile, n1);
            }
            if (tile >= ntiles) break;
            if (at != cti) {
                leave_expert();
                at = cti;
                const int s0 = s.start[at], ns = s.start[at + 1] - s0;
                nt = (ns + 7) / 8;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int q = 8 * t + g;
                    xp[t] = q < ns ? p.h + static_cast<size_t>(s0 + q) * K : nullptr;
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                }
            }
            unit_mma<FMT, ACT, NT>(ring[d], xp, nt, cks * U::SPAN, K, c, acc);
            if (U::ROW_SCALE) {
                f0 = ring[d].scale(0);
                f1 = ring[d].scale(1);
            }
            cks += kFewWarps;
            settle(ctile, cti, cks);
            fetch(ring[d]);
        }
    }
}

template <int FMT, int ACT, int NT>
cudaError_t launch_few_nt(const FewParams& p, int sms, cudaStream_t st) {
    const size_t gu_smem = sizeof(float4) * 2 * kFewWarps * NT * 32;
    const cudaError_t e = launch_pdl(few_gate_up_kernel<FMT, ACT, NT>, sms, kFewThreads, gu_smem, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(few_down_kernel<FMT, ACT, NT>, sms < p.H ? sms : p.H, kFewThreads,
                      sizeof(float) * kFewWarps * p.T * 17, st, p);
}

template <int FMT, int ACT>
cudaError_t launch_few(const FewParams& p, int sms, cudaStream_t st) {
    if (p.T <= 8) return launch_few_nt<FMT, ACT, 1>(p, sms, st);
    if (p.T <= 16) return launch_few_nt<FMT, ACT, 2>(p, sms, st);
    return launch_few_nt<FMT, ACT, 4>(p, sms, st);
}

}  // namespace moe
