// The whole expert layer for at most 32 tokens, in two kernels.
//
//     h[t, j, :] = act( silu(x[t] . Wg_e) * (x[t] . Wu_e) ),  e = ids[t, j]
//     out[t]     = act( sum_j w[t, j] * (h[t, j] . Wd_e) )
//
// With few tokens the layer is bound by the touched experts' weight bytes, and
// at one or two tokens as much by latency, so nothing stands between the
// routing and the weight stream: no sort, no gather, no padding, and no
// separate combine. Both kernels rebuild the same small plan in shared memory
// from the ids (selecting the experts themselves when given logits): a bit
// mask of tokens per expert (T <= 32 bits), the touched experts in ascending
// order and, per expert, its "slots" (distinct tokens, ascending). Each CTA
// takes an equal share of the weight rows, and each of its warps an equal,
// contiguous share of the CTA's units (stream.cuh):
//   gate/up  rows (touched expert, i): 8 gate and the 8 up rows of the same i
//            to a unit, so one lane holds both sums of an h element. A warp
//            finishes an item (8 rows, the whole contraction) by itself; items
//            cut between warps are added once, at the end, in warp order.
//   down     columns [n0, n1) of every touched expert, so the weighted sum
//            over the experts stays inside the CTA: each warp keeps its own
//            f32 sums per token in shared memory and adds an expert's products,
//            times the weight, when it leaves that expert; the warps' sums are
//            added in warp order.
// No atomics on values: results do not depend on timing. The down kernel is
// launched early (programmatic dependent launch): its plan and first weight
// copies need nothing of the gate/up kernel, only the token operand waits.
#pragma once

#include "few_params.cuh"
#include "route_row.cuh"
#include "stream.cuh"

namespace moe {

constexpr int kFewPairs = MOE_MAX_FEW_TOKENS * MOE_MAX_TOPK;

// Warps per CTA and ring stages per warp. bf16 has next to nothing to convert:
// 8 warps keep up, and a CTA of each kernel fits an SM, so the down kernel's
// start hides behind the gate/up kernel's end. The quantised formats are bound
// by the instructions of their conversion and want all the warps of an SM.
template <int FMT> struct FewShape {
    static constexpr int WARPS = FMT == MOE_W_BF16 ? 8 : 15;
    static constexpr int RING = FMT == MOE_W_BF16 ? 7 : (FMT == MOE_W_GPTQ_INT4 ? 8 : 6);
    static constexpr int RESIDENT = FMT == MOE_W_BF16 ? 2 : 1;  // CTAs per SM the registers must allow
};

struct FewPlan {
    int n;                              // touched experts
    int te[MOE_MAX_EXPERTS];            // touched experts, ascending
    int start[MOE_MAX_EXPERTS + 1];     // first slot of each
    uint32_t mask[MOE_MAX_EXPERTS];     // by expert id: tokens routed to it
    int first[MOE_MAX_EXPERTS];         // by expert id: first slot
    int ids[kFewPairs];
    float slot_w[kFewPairs];
    uint8_t slot_tok[kFewPairs];
    uint32_t scan[MOE_MAX_EXPERTS / 32];
};

static __device__ __noinline__ void route_row_nan(const float* lrow, int lane, int E, int k, int renorm, int32_t* ids,
                                           float* w) {
    float v[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) v[j] = lane + 32 * j < E ? lrow[lane + 32 * j] : 0.0f;
    route_row(v, lane, E, k, renorm, ids, w);
}

// Everything of the plan but the weights; THREADS threads, all of them here.
// `publish`: this CTA reports bad ids.
template <int THREADS>
__device__ __forceinline__ void build_plan(FewPlan& s, const FewParams& p, bool publish) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.T * p.k;
    static_assert(THREADS >= MOE_MAX_EXPERTS, "one thread per expert");
    if (tid < MOE_MAX_EXPERTS) s.mask[tid] = 0;
    if (p.logits) {
        for (int t = warp; t < p.T; t += THREADS / 32) {
            const float* lrow = p.logits + t * p.E;
            float v[kPerLane], sv;
            int si;
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) v[j] = lane + 32 * j < p.E ? __ldg(lrow + lane + 32 * j) : 0.0f;
            if (!select_row(v, lane, p.E, p.k, sv, si)) {
                route_row_nan(lrow, lane, p.E, p.k, p.renorm, s.ids + t * p.k, s.slot_w);  // slot_w: scratch here
                continue;
            }
            if (lane < p.k) s.ids[t * p.k + lane] = si;
        }
    } else {
        for (int i = tid; i < P; i += THREADS) s.ids[i] = p.ids[i];
    }
    __syncthreads();
    for (int i = tid; i < P; i += THREADS) {
        const int e = s.ids[i];
        if (e >= 0 && e < p.E) atomicOr(&s.mask[e], 1u << (i / p.k));
        else if (publish) set_err(p.err, MOE_DEV_ERR_EXPERT_ID);
    }
    __syncthreads();
    // prefix sums over the experts: touched experts in the high half, slots in the low
    uint32_t m = 0, mine = 0, inc = 0;
    if (tid < MOE_MAX_EXPERTS) {
        m = s.mask[tid];
        inc = mine = (m ? 1u << 16 : 0u) + __popc(m);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) s.scan[warp] = inc;
    }
    __syncthreads();
    if (tid < MOE_MAX_EXPERTS) {
        uint32_t before = inc - mine;
        for (int w = 0; w < warp; ++w) before += s.scan[w];
        if (m) {
            s.te[before >> 16] = tid;
            s.start[before >> 16] = before & 0xffffu;
            s.first[tid] = before & 0xffffu;
        }
        if (tid == MOE_MAX_EXPERTS - 1) {
            const uint32_t all = before + mine;
            s.n = all >> 16;
            s.start[all >> 16] = all & 0xffffu;
        }
    }
    __syncthreads();
    for (int i = tid; i < P; i += THREADS) {
        const int e = s.ids[i], t = i / p.k;
        if (e >= 0 && e < p.E)
            s.slot_tok[s.first[e] + __popc(s.mask[e] & ((1u << t) - 1u))] = static_cast<uint8_t>(t);
    }
    __syncthreads();
}

// The slots' weights, from the weights in global memory: an expert that a token
// names twice gets the sum.
template <int THREADS> __device__ __forceinline__ void slot_weights(FewPlan& s, const FewParams& p) {
    const int P = p.T * p.k;
    for (int i = threadIdx.x; i < P; i += THREADS) {
        const int e = s.ids[i], t = i / p.k, end = (t + 1) * p.k;
        if (e < 0 || e >= p.E) continue;
        bool again = false;
        for (int j = t * p.k; j < i; ++j) again |= s.ids[j] == e;
        if (again) continue;
        float w = p.weights[i];
        for (int j = i + 1; j < end; ++j)
            if (s.ids[j] == e) w += p.weights[j];
        s.slot_w[s.first[e] + __popc(s.mask[e] & ((1u << t) - 1u))] = w;
    }
}

// One warp: ids and weights of the routing outputs' rows t, t + step, ...
__device__ __forceinline__ void publish_routing(const FewParams& p, int t, int step, int lane) {
    for (; t < p.T; t += step) {
        const float* lrow = p.logits + t * p.E;
        float v[kPerLane], sv;
        int si;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) v[j] = lane + 32 * j < p.E ? __ldg(lrow + lane + 32 * j) : 0.0f;
        if (select_row(v, lane, p.E, p.k, sv, si))
            finish_row(v, lane, p.E, p.k, p.renorm, __shfl_sync(0xffffffffu, sv, 0), sv, si, p.ids + t * p.k,
                       p.weights + t * p.k);
        else
            route_row_nan(lrow, lane, p.E, p.k, p.renorm, p.ids + t * p.k, p.weights + t * p.k);
    }
}

// ---- gate/up ----------------------------------------------------------------------

template <int FMT, int ACT, int NT>
__global__ void __launch_bounds__((FewShape<FMT>::WARPS + 1) * 32, FewShape<FMT>::RESIDENT)
few_gate_up_kernel(const FewParams p) {
    using U = Unit<FMT, ACT>;
    using S = Stage<U>;
    constexpr int RING = FewShape<FMT>::RING, W = FewShape<FMT>::WARPS;
    extern __shared__ uint8_t few_smem[];
    float4* cut = reinterpret_cast<float4*>(few_smem + W * RING * S::BYTES);  // [W][2][NT][32]: sums of cut items
    __shared__ FewPlan s;
    pdl_wait();
    pdl_launch_next();
    build_plan<(W + 1) * 32>(s, p, blockIdx.x == 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    if (warp == W) {  // beside the products: the routing outputs, one row per CTA
        if (p.logits) publish_routing(p, blockIdx.x, gridDim.x, lane);
        __syncthreads();
        return;
    }
    const int I = p.I, K = p.H;
    const int64_t rows = static_cast<int64_t>(s.n) * I;  // row = touched index * I + i
    const int r0 = static_cast<int>(rows * blockIdx.x / gridDim.x);
    const int r1 = static_cast<int>(rows * (blockIdx.x + 1) / gridDim.x);
    const int nk = (K + U::SPAN - 1) / U::SPAN;
    // items: up to 8 consecutive rows of one expert
    const int ti0 = r0 / I, i0 = r0 - ti0 * I, per = (I + 7) / 8;
    const int f_rows = min(r1 - r0, I - i0), f_items = (f_rows + 7) / 8;
    const int rest = r1 - r0 - f_rows, last = rest % I;
    const int64_t units = static_cast<int64_t>(f_items + rest / I * per + (last + 7) / 8) * nk;
    auto first_unit = [&](int w) { return static_cast<int>(units * w / W); };
    auto locate = [&](int q, int& ti, int& i) {  // item q of the CTA
        if (q < f_items) {
            ti = ti0;
            i = i0 + 8 * q;
        } else {
            ti = ti0 + 1 + (q - f_items) / per;
            i = 8 * ((q - f_items) % per);
        }
    };
    auto row_end = [&](int ti) { return min(I, r1 - ti * I); };
    const int u0 = first_unit(warp), u1 = first_unit(warp + 1);
    uint8_t* ring = few_smem + warp * RING * S::BYTES;

    // where the copies are
    int lleft = u1 - u0, lks = u0 % nk, lti, li;
    bool laim = true;
    locate(u0 / nk, lti, li);
    typename U::Src src;
    const uint16_t* lx = nullptr;
    auto fetch = [&](int stage) {
        if (lleft > 0) {
            if (laim) {
                const WBase b = expert_base<FMT>(p.gu.w, p.gu.scales, p.gu.zeros, 2 * I, K, p.gu.group_size, s.te[lti]);
                const int cnt = min(8, row_end(lti) - li);
                src.aim(b, UnitRows{li, cnt, I + li, cnt}, lane);
                if (U::X_RING) {
                    const int slot = s.start[lti] + g;
                    lx = slot < s.start[lti + 1] ? p.x + static_cast<size_t>(s.slot_tok[slot]) * K + U::k_of(0, c)
                                                 : nullptr;
                }
                laim = false;
            }
            uint8_t* st = ring + stage * S::BYTES;
            const int k0 = lks * U::SPAN;
            const bool tail = k0 + U::SPAN > K;
            src.load(st, k0, K, tail, lane);
            if (U::X_RING) Tokens<U>::copy(st + S::X_AT, lx, k0, K, tail, lane);
            --lleft;
            if (++lks == nk) {
                lks = 0;
                laim = true;
                li += 8;
                if (li >= row_end(lti)) {
                    li = 0;
                    ++lti;
                }
            }
        }
        cp_async_commit();
    };
    for (int d = 0; d < RING - 1; ++d) fetch(d);

    // writes the h elements of an item's finished sums
    auto finish = [&](const float (&acc)[NT][4], int ti, int i) {
        const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, e = s.te[ti];
        if (i + g >= row_end(ti)) return;
        const float gs2 = FMT == MOE_W_NVFP4 ? __ldg(p.gu.scale2 + e) : 1.0f;
        const float us2 = FMT == MOE_W_NVFP4 ? __ldg(p.gu.scale2 + p.E + e) : 1.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int slot = 8 * t + 2 * c + q;
                if (slot < ns) {
                    const float gs = gs2 * acc[t][q], us = us2 * acc[t][2 + q];
                    const float v = __fdividef(gs, 1.0f + __expf(-gs)) * us;
                    reinterpret_cast<typename Act<ACT>::T*>(p.h)[static_cast<size_t>(s0 + slot) * I + i + g] =
                        Act<ACT>::from_f(v);
                }
            }
    };

    float acc[NT][4];
    int left = u1 - u0, ks = u0 % nk, stage = 0, ti, i;
    locate(u0 / nk, ti, i);
    while (left > 0) {
        const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, nt = (ns + 7) / 8;
        const int cnt = min(8, row_end(ti) - i), begin = ks, end = min(nk, ks + left);
        const UnitRows rows_u{i, cnt, I + i, cnt};
        const uint16_t* xp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int q = 8 * t + g;
            xp[t] = q < ns ? p.x + static_cast<size_t>(s.slot_tok[s0 + q]) * K + U::k_of(0, c) : nullptr;
            acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
        }
        float f0 = 1.0f, f1 = 1.0f;
        if (U::ROW_SCALE && g < cnt) {
            const float* sc = static_cast<const float*>(p.gu.scales) + static_cast<size_t>(2 * I) * s.te[ti] + i + g;
            f0 = __ldg(sc);
            f1 = __ldg(sc + I);
        }
        for (; ks < end; ++ks) {
            const int k0 = ks * U::SPAN;
            const bool tail = k0 + U::SPAN > K;
            Tokens<U> x;
            if (!U::X_RING) x.fetch(xp[0], k0, K, tail, lane);
            __syncwarp();  // every lane is done with the stage refilled now
            fetch(stage == 0 ? RING - 1 : stage - 1);
            cp_async_wait_group<RING - 1>();
            __syncwarp();  // scales were copied by other lanes
            const uint8_t* st = ring + stage * S::BYTES;
            U u;
            u.open(st, rows_u, lane);
            if (U::X_RING) x.open(st + S::X_AT, xp[0], lane);
            unit_mma<U, ACT, NT>(u, x, xp, nt, k0, K, tail, lane, acc);
            if (++stage == RING) stage = 0;
        }
        left -= end - begin;
        if (U::ROW_SCALE) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                acc[t][0] *= f0;
                acc[t][1] *= f0;
                acc[t][2] *= f1;
                acc[t][3] *= f1;
            }
        }
        if (begin == 0 && end == nk) {
            finish(acc, ti, i);
        } else {
            float4* dst = cut + (warp * 2 + (begin == 0)) * NT * 32 + lane;
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < nt) dst[t * 32] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        }
        ks = 0;
        i += 8;
        if (i >= row_end(ti)) {
            i = 0;
            ++ti;
        }
    }
    __syncthreads();
    // The items cut between warps: the first warp that starts inside an item adds
    // its parts in warp order, from the warp before (where the item begins) on.
    if (warp == 0 || u0 >= units || u0 % nk == 0 || first_unit(warp - 1) > u0 / nk * nk) return;
    const int q = u0 / nk, q_end = (q + 1) * nk;
    locate(q, ti, i);
    const int nt = (s.start[ti + 1] - s.start[ti] + 7) / 8;
    const float4* src0 = cut + ((warp - 1) * 2 + 1) * NT * 32 + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float4 v = t < nt ? src0[t * 32] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        acc[t][0] = v.x;
        acc[t][1] = v.y;
        acc[t][2] = v.z;
        acc[t][3] = v.w;
    }
    for (int w = warp; w < W; ++w) {
        const int from = first_unit(w), to = first_unit(w + 1);
        if (from >= q_end) break;
        if (from == to) continue;
        const float4* more = cut + w * 2 * NT * 32 + lane;
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t < nt) {
                const float4 v = more[t * 32];
                acc[t][0] += v.x;
                acc[t][1] += v.y;
                acc[t][2] += v.z;
                acc[t][3] += v.w;
            }
    }
    finish(acc, ti, i);
}

// ---- down ---------------------------------------------------------------------------

// The end of a 16-column tile: adds the warps' sums in warp order, writes the
// columns and clears the sums for the next tile.
template <int ACT, int W>
__device__ __noinline__ void few_tile_end(float* sums, uint16_t* out, int T, int H, int n0, int n1) {
    __syncthreads();
    for (int i = threadIdx.x; i < T * 16; i += W * 32) {
        const int tok = i >> 4, col = i & 15;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
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
__global__ void __launch_bounds__(FewShape<FMT>::WARPS * 32, FewShape<FMT>::RESIDENT)
few_down_kernel(const FewParams p) {
    using U = Unit<FMT, ACT>;
    using S = Stage<U>;
    constexpr int RING = FewShape<FMT>::RING, W = FewShape<FMT>::WARPS;
    extern __shared__ uint8_t few_smem[];
    float* sums = reinterpret_cast<float*>(few_smem + W * RING * S::BYTES);  // [W][T][17]: sums of 16 columns
    __shared__ FewPlan s;
    // before the wait: only what was complete before the gate/up kernel started
    // (logits, or ids given as inputs) and the weights
    build_plan<W * 32>(s, p, false);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int K = p.I, n = s.n;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.H) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.H) * (blockIdx.x + 1) / gridDim.x);
    const int ntiles = (n1 - n0 + 15) / 16;
    const int nks = (K + U::SPAN - 1) / U::SPAN;
    float* mine = sums + warp * p.T * 17;
    for (int i = tid; i < W * p.T * 17; i += W * 32) sums[i] = 0.0f;

    // A tile's units (touched expert, contraction step): this warp's share is the same in every tile
    const int64_t units = static_cast<int64_t>(n) * nks;
    const int u0 = static_cast<int>(units * warp / W), count = static_cast<int>(units * (warp + 1) / W) - u0;
    const int ti_first = u0 / nks, ks_first = u0 - ti_first * nks;
    uint8_t* ring = few_smem + warp * RING * S::BYTES;

    // where the copies are
    int ltile = count > 0 ? 0 : ntiles, lti = ti_first, lks = ks_first, lleft = count;
    bool laim = true;
    typename U::Src src;
    auto fetch_w = [&](int stage) {
        if (laim) {
            const WBase b = expert_base<FMT>(p.down.w, p.down.scales, p.down.zeros, p.H, K, p.down.group_size, s.te[lti]);
            const int a = n0 + 16 * ltile;
            src.aim(b, UnitRows{a, n1 - a, a + 8, n1 - a - 8}, lane);
            laim = false;
        }
        const int k0 = lks * U::SPAN;
        src.load(ring + stage * S::BYTES, k0, K, k0 + U::SPAN > K, lane);
    };
    auto fetch_h = [&](int stage, int ti, int ks) {
        const int slot = s.start[ti] + g, k0 = ks * U::SPAN;
        Tokens<U>::copy(ring + stage * S::BYTES + S::X_AT,
                        slot < s.start[ti + 1] ? p.h + static_cast<size_t>(slot) * K + U::k_of(0, c) : nullptr, k0, K,
                        k0 + U::SPAN > K, lane);
    };
    auto advance = [&]() {
        if (++lks == nks) {
            lks = 0;
            ++lti;
            laim = true;
        }
        if (--lleft == 0) {
            ++ltile;
            lti = ti_first;
            lks = ks_first;
            lleft = count;
            laim = true;
        }
    };
    for (int d = 0; d < RING - 1 && ltile < ntiles; ++d) {
        fetch_w(d);
        advance();
    }
    pdl_wait();  // h and the routing outputs are complete
    slot_weights<W * 32>(s, p);
    {
        int tile = count > 0 ? 0 : ntiles, ti = ti_first, ks = ks_first, left = count;
        for (int d = 0; d < RING - 1; ++d) {
            if (U::X_RING && tile < ntiles) {
                fetch_h(d, ti, ks);
                if (++ks == nks) {
                    ks = 0;
                    ++ti;
                }
                if (--left == 0) {
                    ++tile;
                    ti = ti_first;
                    ks = ks_first;
                    left = count;
                }
            }
            cp_async_commit();
        }
    }
    __syncthreads();  // the slots' weights, and the sums are zero

    float acc[NT][4];
    int stage = 0;
    for (int tile = 0; tile < ntiles; ++tile) {
        const int a = n0 + 16 * tile;
        const UnitRows rows_u{a, n1 - a, a + 8, n1 - a - 8};
        int left = count, ti = ti_first, ks = ks_first;
        while (left > 0) {  // one expert's units
            const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, nt = (ns + 7) / 8, e = s.te[ti];
            const int end = min(nks, ks + left);
            left -= end - ks;
            const uint16_t* xp[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int q = 8 * t + g;
                xp[t] = q < ns ? p.h + static_cast<size_t>(s0 + q) * K + U::k_of(0, c) : nullptr;
                acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
            }
            float f0 = 1.0f, f1 = 1.0f;
            if (U::ROW_SCALE) {
                const float* sc = static_cast<const float*>(p.down.scales) + static_cast<size_t>(p.H) * e + a + g;
                f0 = a + g < n1 ? __ldg(sc) : 0.0f;
                f1 = a + 8 + g < n1 ? __ldg(sc + 8) : 0.0f;
            }
            if (FMT == MOE_W_NVFP4) f0 = f1 = __ldg(p.down.scale2 + e);
            for (; ks < end; ++ks) {
                const int k0 = ks * U::SPAN;
                const bool tail = k0 + U::SPAN > K;
                Tokens<U> x;
                if (!U::X_RING) x.fetch(xp[0], k0, K, tail, lane);
                __syncwarp();  // every lane is done with the stage refilled now
                if (ltile < ntiles) {
                    const int st = stage == 0 ? RING - 1 : stage - 1;
                    fetch_w(st);
                    if (U::X_RING) fetch_h(st, lti, lks);
                    advance();
                }
                cp_async_commit();
                cp_async_wait_group<RING - 1>();
                __syncwarp();  // scales were copied by other lanes
                const uint8_t* st = ring + stage * S::BYTES;
                U u;
                u.open(st, rows_u, lane);
                if (U::X_RING) x.open(st + S::X_AT, xp[0], lane);
                unit_mma<U, ACT, NT>(u, x, xp, nt, k0, K, tail, lane, acc);
                if (++stage == RING) stage = 0;
            }
            // leave the expert: add its products, times the weights, to the tokens' sums
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t > 0 && t >= nt) break;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int slot = 8 * t + 2 * c + q;
                    if (slot < ns) {
                        float* dst = mine + s.slot_tok[s0 + slot] * 17 + g;
                        const float w = s.slot_w[s0 + slot];
                        dst[0] = fmaf(w, f0 * acc[t][q], dst[0]);
                        dst[8] = fmaf(w, f1 * acc[t][2 + q], dst[8]);
                    }
                }
            }
            __syncwarp();  // another lane adds to the same token's sums for the next expert
            ks = 0;
            ++ti;
        }
        few_tile_end<ACT, W>(sums, p.out, p.T, p.H, a, n1);
    }
}

template <int FMT, int ACT, int NT>
cudaError_t launch_few_nt(const FewParams& p, int sms, cudaStream_t st) {
    constexpr int W = FewShape<FMT>::WARPS;
    constexpr int ring = W * FewShape<FMT>::RING * Stage<Unit<FMT, ACT>>::BYTES;
    constexpr int gu_smem = ring + static_cast<int>(sizeof(float4)) * 2 * W * NT * 32;
    constexpr int dn_most = ring + static_cast<int>(sizeof(float)) * W * 8 * NT * 17;
    static int configured_for = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        if (set_smem_limit(reinterpret_cast<const void*>(few_gate_up_kernel<FMT, ACT, NT>), gu_smem) != MOE_OK ||
            set_smem_limit(reinterpret_cast<const void*>(few_down_kernel<FMT, ACT, NT>), dn_most) != MOE_OK)
            return cudaGetLastError();
        configured_for = dev;
    }
    const cudaError_t e = launch_pdl(few_gate_up_kernel<FMT, ACT, NT>, sms, (W + 1) * 32, gu_smem, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(few_down_kernel<FMT, ACT, NT>, sms < p.H ? sms : p.H, W * 32,
                      ring + sizeof(float) * W * p.T * 17, st, p);
}

template <int FMT, int ACT>
cudaError_t launch_few(const FewParams& p, int sms, cudaStream_t st) {
    if (p.T <= 8) return launch_few_nt<FMT, ACT, 1>(p, sms, st);
    if (p.T <= 16) return launch_few_nt<FMT, ACT, 2>(p, sms, st);
    return launch_few_nt<FMT, ACT, 4>(p, sms, st);
}

}  // namespace moe
