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
// order and, per expert, its "slots" (distinct tokens, ascending). An expert
// with more slots than a unit's product takes (8 or 16) is listed again for
// the rest, and its weights read again. Each CTA takes an equal share of the
// weight rows, and each of its warps an equal, contiguous share of the CTA's
// units (stream.cuh):
//   gate/up  rows (touched expert, i): gate rows and the up rows of the same i
//            to a unit, so one lane holds both sums of an h element. A warp
//            finishes an item (16 or 32 such rows, the whole contraction) by
//            itself; items cut between warps are added once, at the end, in
//            warp order.
//   down     a cluster of 2, 4 or 8 CTAs takes columns [n0, n1) of every
//            touched expert, so the weighted sum over the experts stays inside
//            the cluster: each warp keeps its own f32 sums per token in shared
//            memory and adds an expert's products, times the weight, when it
//            leaves that expert; the warps' sums are added in warp order, and
//            the CTAs' in rank order through distributed shared memory. A unit
//            has 32 columns, so narrow layers take larger clusters: T = 16,
//            H = 256, I = 7000, 8 bf16 experts 29.4 us in clusters of 8, 51.6 in
//            pairs (4 columns each); at H = 2048 pairs have 27 columns, and one
//            CTA per column share had 13.
// Measured, us and of the touched weights' time at HBM's rate: bf16, 8 of 128
// experts of 2048 x 768, one token 23.4 (47%: 4.9 pass before the first weights
// arrive, about 4 between the kernels and at the end); 8 experts of 4096 x 14336,
// 7 tokens 410 (88%, HBM); GPTQ, 64 of 2048 x 1408, 16 tokens 82 (41%) and NVFP4,
// 128 of 2048 x 768, 32 tokens 113 (39%): the conversion keeps 50 and 60% of the
// issue slots and 45 and 54% of the integer pipe busy over the whole kernels,
// starts and ends included. (Gate/up on pairs of CTAs too: GPTQ 82.4 -> 85.8.)
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
// by the instructions of their conversion and want all the warps of an SM (us at
// 15 / 11 warps, T = 32, H = 2048: FP8 110 / 120, NVFP4 111 / 115; GPTQ, T = 16,
// 84 / 87). GPTQ with two token tiles has 11, which is what shared memory holds.
// A fifth stage is worth 1% to FP8, and the others have no room for it.
template <int FMT, int NT> struct FewShape {
    static constexpr bool DENSE = FMT == MOE_W_BF16, GPTQ = FMT == MOE_W_GPTQ_INT4;
    static constexpr int WARPS = DENSE ? 8 : (GPTQ && NT > 1 ? 11 : 15);
    static constexpr int GU_RING = FMT == MOE_W_FP8_E4M3 ? 5 : 4;
    static constexpr int DN_RING = 4;
    static constexpr int RESIDENT = DENSE ? 2 : 1;  // CTAs per SM the registers must allow
};
constexpr int kFewEntries = MOE_MAX_EXPERTS + kFewPairs / 8;
constexpr int kFewCols = 33;  // columns of a down tile, and a pad
constexpr int kFewMaxLg = 3, kFewMaxCluster = 1 << kFewMaxLg;  // CTAs that share a down tile, at most

struct FewPlan {
    int n;                           // entries: touched experts, ascending, split
    int te[kFewEntries];             // expert of each
    int start[kFewEntries + 1];      // first slot of each
    uint32_t mask[MOE_MAX_EXPERTS / 8 * 9];  // by expert id (at(id)): tokens routed to it
    int first[MOE_MAX_EXPERTS / 8 * 9];      // by expert id: first slot
    float slot_w[kFewPairs];
    uint8_t slot_tok[kFewPairs];
    // eight ids and a pad: the scan reads eight consecutive ones a lane
    static __device__ __forceinline__ int at(int id) { return id + (id >> 3); }
    // the slot of token t with expert id
    __device__ __forceinline__ int slot_of(int id, int t) const {
        return first[at(id)] + __popc(mask[at(id)] & ((1u << t) - 1u));
    }
};

// [x0, x1): part i of n nearly equal parts of [0, all)
__device__ __forceinline__ void part_of(int all, int n, int i, int& x0, int& x1) {
    const int q = all / n, r = all - q * n;
    x0 = q * i + min(i, r);
    x1 = x0 + q + (i < r ? 1 : 0);
}

static __device__ __noinline__ void route_row_nan(const float* lrow, int lane, int E, int k, int renorm, int32_t* ids,
                                                  float* w) {
    float v[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) v[j] = lane + 32 * j < E ? lrow[lane + 32 * j] : 0.0f;
    route_row(v, lane, E, k, renorm, ids, w);
}

// Everything of the plan but the weights; WARPS warps, all of them here; at
// most SLOTS slots an entry. A warp takes tokens warp, warp + WARPS, ..., and
// lane j < k of it the token's pair j: the experts are selected from the
// logits (`select`) or read. `publish`: this CTA reports bad ids. The plan is
// on the way of every weight load, so it is short: four barriers, no division.
template <int WARPS, int SLOTS>
__device__ __forceinline__ void build_plan(FewPlan& s, const FewParams& p, bool select, bool publish) {
    constexpr int ROUNDS = (MOE_MAX_FEW_TOKENS + WARPS - 1) / WARPS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int MASKS = MOE_MAX_EXPERTS / 8 * 9;
    for (int i = tid; i < MASKS; i += WARPS * 32) s.mask[i] = 0;
    __syncthreads();
    int ids[ROUNDS];
    const int mine_n = (p.T - warp + WARPS - 1) / WARPS;  // this warp's tokens
    if (select) {
        const float* lrow[ROUNDS];
        float sv[ROUNDS];
#pragma unroll
        for (int q = 0; q < ROUNDS; ++q) lrow[q] = p.logits + (warp + q * WARPS) * p.E;
        uint32_t nan = 0;
        if (mine_n == 1) {
            const float* one[1] = {lrow[0]};
            float v[1];
            int id[1];
            nan = select_rows<1>(one, 1, lane, p.E, p.k, v, id);
            ids[0] = id[0];
        } else if (mine_n > 1) {
            nan = select_rows<ROUNDS>(lrow, mine_n, lane, p.E, p.k, sv, ids);
        }
        for (; nan; nan &= nan - 1) {
            const int bad = __ffs(nan) - 1, t = warp + bad * WARPS;
            // into scratch of the token's and the warp's own (slot_w and te are filled later)
            int32_t* scratch = reinterpret_cast<int32_t*>(s.slot_w) + t * MOE_MAX_TOPK;
            route_row_nan(p.logits + t * p.E, lane, p.E, p.k, p.renorm, scratch,
                          reinterpret_cast<float*>(s.te) + warp * MOE_MAX_TOPK);
            __syncwarp();
#pragma unroll
            for (int q = 0; q < ROUNDS; ++q)
                if (q == bad && lane < p.k) ids[q] = scratch[lane];
        }
    }
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        const int t = warp + q * WARPS;
        if (!select && q < mine_n && lane < p.k) {
            ids[q] = p.ids[t * p.k + lane];
            if (publish && (ids[q] < 0 || ids[q] >= p.E)) set_err(p.err, MOE_DEV_ERR_EXPERT_ID);
        }
        if (q >= mine_n || lane >= p.k || ids[q] < 0 || ids[q] >= p.E) ids[q] = -1;
        else atomicOr(&s.mask[s.at(ids[q])], 1u << t);
    }
    __syncthreads();
    if (warp == 0) {
        // prefix sums over the experts, eight consecutive ones a lane: entries in the high half, slots in the low
        uint32_t cnt[8], mine = 0;
        bool many = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) cnt[j] = s.mask[lane * 9 + j];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cnt[j] = __popc(cnt[j]);
            many |= cnt[j] > SLOTS;
            mine += ((cnt[j] + SLOTS - 1) / SLOTS << 16) + cnt[j];
        }
        uint32_t inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        uint32_t at = inc - mine;
        if (!__any_sync(0xffffffffu, many)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s.first[lane * 9 + j] = at & 0xffffu;
                if (cnt[j]) {
                    s.te[at >> 16] = lane * 8 + j;
                    s.start[at >> 16] = at & 0xffffu;
                    at += (1u << 16) + cnt[j];
                }
            }
        } else {
            for (int j = 0; j < 8; ++j) {
                s.first[lane * 9 + j] = at & 0xffffu;
                const uint32_t n = __popc(s.mask[lane * 9 + j]);
                for (uint32_t c = 0; c < n; c += SLOTS) {
                    s.te[at >> 16] = lane * 8 + j;
                    s.start[at >> 16] = at & 0xffffu;
                    at += (1u << 16) + min(n - c, static_cast<uint32_t>(SLOTS));
                }
            }
        }
        if (lane == 31) {
            s.n = inc >> 16;
            s.start[inc >> 16] = inc & 0xffffu;
        }
    }
    static_assert(MOE_MAX_EXPERTS == 256, "eight experts a lane");
    __syncthreads();
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q)
        if (ids[q] >= 0) s.slot_tok[s.slot_of(ids[q], warp + q * WARPS)] = static_cast<uint8_t>(warp + q * WARPS);
    __syncthreads();
}

// The slots' weights, from the ids and weights in global memory: an expert that
// a token names twice gets the sum, in the order of its pairs.
template <int WARPS> __device__ __forceinline__ void slot_weights(FewPlan& s, const FewParams& p) {
    const int lane = threadIdx.x & 31;
    for (int t = threadIdx.x >> 5; t < p.T; t += WARPS) {
        const int e = lane < p.k ? p.ids[t * p.k + lane] : -1;
        const float w = lane < p.k ? p.weights[t * p.k + lane] : 0.0f;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        float sum = 0.0f;
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            if (same >> j & 1) sum = j == __ffs(same) - 1 ? wj : sum + wj;
        }
        if (lane < p.k && e >= 0 && e < p.E && lane == __ffs(same) - 1)
            s.slot_w[s.slot_of(e, t)] = sum;
    }
}

// One warp: ids and weights of the routing outputs' rows t, t + step, ...
__device__ __forceinline__ void publish_routing(const FewParams& p, int t, int step, int lane) {
    for (; t < p.T; t += step) {
        const float* lrow[1] = {p.logits + t * p.E};
        float v[kPerLane], sv[1];
        int si[1];
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) v[j] = lane + 32 * j < p.E ? __ldg(lrow[0] + lane + 32 * j) : 0.0f;
        if (select_rows<1>(lrow, 1, lane, p.E, p.k, sv, si) == 0)
            finish_row(v, lane, p.E, p.k, p.renorm, __shfl_sync(0xffffffffu, sv[0], 0), sv[0], si[0], p.ids + t * p.k,
                       p.weights + t * p.k);
        else
            route_row_nan(lrow[0], lane, p.E, p.k, p.renorm, p.ids + t * p.k, p.weights + t * p.k);
    }
}

// ---- gate/up ----------------------------------------------------------------------

template <int FMT, int ACT, int NT>
__global__ void __launch_bounds__((FewShape<FMT, NT>::WARPS + 1) * 32, FewShape<FMT, NT>::RESIDENT)
few_gate_up_kernel(const FewParams p) {
    using U = Unit<FMT, ACT, true>;
    using S = Stage<U>;
    constexpr int RING = FewShape<FMT, NT>::GU_RING, W = FewShape<FMT, NT>::WARPS, MT = U::MT, ROWS = U::ROWS;
    extern __shared__ uint8_t few_smem[];
    float4* cut = reinterpret_cast<float4*>(few_smem + W * RING * S::BYTES);  // [W][2][MT][NT][32]: sums of cut items
    __shared__ FewPlan s;
    pdl_wait();
    pdl_launch_next();  // not before the wait: the down kernel reads the routing before its own
    build_plan<W + 1, 8 * NT>(s, p, p.logits != nullptr, blockIdx.x == 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    if (warp == W) {  // beside the products: the routing outputs, one row per CTA
        if (p.logits) publish_routing(p, blockIdx.x, gridDim.x, lane);
        __syncthreads();
        return;
    }
    const int I = p.I, K = p.H;
    // The CTA's rows, row = entry * I + i. Where items are many, shares of whole
    // items: the quantised formats take as long for part of one.
    const int whole = !FewShape<FMT, NT>::DENSE && I % ROWS == 0 && s.n * (I / ROWS) >= 8 * static_cast<int>(gridDim.x);
    const int align = whole ? ROWS : U::ALIGN;
    int r0, r1;
    part_of(s.n * (I / align), gridDim.x, blockIdx.x, r0, r1);
    r0 *= align;
    r1 *= align;
    const int nk = (K + U::SPAN - 1) / U::SPAN;
    // items: up to ROWS consecutive rows of one entry
    const int ti0 = r0 / I, i0 = r0 - ti0 * I, per = (I + ROWS - 1) / ROWS;
    const int f_rows = min(r1 - r0, I - i0), f_items = (f_rows + ROWS - 1) / ROWS;
    const int rest = r1 - r0 - f_rows;
    const int full = rest / I, units = (f_items + full * per + (rest - full * I + ROWS - 1) / ROWS) * nk;
    auto first_unit = [&](int w) { return units / W * w + min(w, units % W); };
    auto locate = [&](int q, int& ti, int& i) {  // item q of the CTA
        if (q < f_items) {
            ti = ti0;
            i = i0 + ROWS * q;
        } else {
            const int e = (q - f_items) / per;
            ti = ti0 + 1 + e;
            i = ROWS * (q - f_items - e * per);
        }
    };
    auto row_end = [&](int ti) { return min(I, r1 - ti * I); };
    auto next_item = [&](int& ti, int& i) {
        i += ROWS;
        if (i >= row_end(ti)) {
            i = 0;
            ++ti;
        }
    };
    const int u0 = first_unit(warp), u1 = first_unit(warp + 1);
    uint8_t* ring = few_smem + warp * RING * S::BYTES;

    const int q0 = u0 / nk, ks0 = u0 - q0 * nk;  // where the share begins: item, contraction step
    int ti, i;
    locate(q0, ti, i);
    // The copies: units left in the warp's share and in the item, contraction
    // indices to its end
    int l_left = u1 - u0, l_item = 0, l_k = ks0 * U::SPAN, l_kleft = 0, lti = ti, li = i;
    typename U::Src src;
    const uint16_t* lx = nullptr;
    bool l_has = false;
    auto fetch = [&](int stage) {
        if (l_left > 0) {
            if (l_item == 0) {
                const WBase b = expert_base<FMT>(p.gu.w, p.gu.scales, p.gu.zeros, 2 * I, K, p.gu.group_size, s.te[lti]);
                const int cnt = min(ROWS, row_end(lti) - li);
                src.aim(b, li, cnt, I + li, cnt, l_k, lane);
                l_kleft = K - l_k;
                l_item = (l_kleft + U::SPAN - 1) / U::SPAN;
                if (U::X_RING) {
                    const int slot = s.start[lti] + g;
                    l_has = slot < s.start[lti + 1];
                    if (l_has) lx = p.x + static_cast<size_t>(s.slot_tok[slot]) * K + l_k + U::k_of(0, c);
                }
                l_k = 0;
                next_item(lti, li);
            }
            uint8_t* st = ring + stage * S::BYTES;
            if (l_kleft >= U::SPAN) src.load(st, lane);
            else src.load_tail(st, l_kleft, lane);
            src.step();
            if (U::X_RING) {
                Tokens<U>::copy(st + S::X_AT, lx, l_has, l_kleft, lane);
                lx += U::SPAN;
            }
            l_kleft -= U::SPAN;
            --l_item;
            --l_left;
        }
        cp_async_commit();
    };
    for (int d = 0; d < RING - 1; ++d) fetch(d);

    // writes the h elements of an item's finished sums
    auto finish = [&](const float (&acc)[MT][NT][4], int ti, int i) {
        const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, e = s.te[ti], end = row_end(ti);
        const float gs2 = FMT == MOE_W_NVFP4 ? U::SCALE_UP * __ldg(p.gu.scale2 + e) : 1.0f;
        const float us2 = FMT == MOE_W_NVFP4 ? U::SCALE_UP * __ldg(p.gu.scale2 + p.E + e) : 1.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = i + U::row_a(m, g);
            if (row >= end) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int slot = 8 * t + 2 * c + q;
                    if (slot < ns) {
                        const float gs = gs2 * acc[m][t][q], us = us2 * acc[m][t][2 + q];
                        const float v = __fdividef(gs, 1.0f + __expf(-gs)) * us;
                        reinterpret_cast<typename Act<ACT>::T*>(p.h)[static_cast<size_t>(s0 + slot) * I + row] =
                            Act<ACT>::from_f(v);
                    }
                }
        }
    };

    float acc[MT][NT][4];
    int left = u1 - u0, ks = ks0, stage = 0;
    while (left > 0) {
        const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, nt = NT > 1 && ns > 8 ? 2 : 1;
        const int end = row_end(ti), begin = ks, stop = min(nk, ks + left);
        const bool has = g < ns, has1 = NT > 1 && 8 + g < ns;
        const uint16_t* x0 = p.x + ks * U::SPAN + U::k_of(0, c);
        const uint16_t* x1 = has1 ? x0 + static_cast<size_t>(s.slot_tok[s0 + 8 + g]) * K : x0;
        if (has) x0 += static_cast<size_t>(s.slot_tok[s0 + g]) * K;
        Tokens<U> x;
        x.clear();
        float f[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            f[m][0] = f[m][1] = 1.0f;
            if (U::ROW_SCALE && i + U::row_a(m, g) < end) {
                const float* sc =
                    static_cast<const float*>(p.gu.scales) + static_cast<size_t>(2 * I) * s.te[ti] + i + U::row_a(m, g);
                f[m][0] = __ldg(sc);
                f[m][1] = __ldg(sc + I);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t][0] = acc[m][t][1] = acc[m][t][2] = acc[m][t][3] = 0.0f;
        }
        int kleft = K - ks * U::SPAN;
        for (; ks < stop; ++ks) {
            if (!U::X_RING) x.fetch(x0, has, kleft, lane);
            __syncwarp();  // every lane is done with the stage refilled now
            fetch(stage == 0 ? RING - 1 : stage - 1);
            cp_async_wait_group<RING - 1>();
            __syncwarp();  // scales were copied by other lanes
            const uint8_t* st = ring + stage * S::BYTES;
            if (++stage == RING) stage = 0;
            U u;
            u.open(st, i, I + i, lane);
            if (U::X_RING) x.open(st + S::X_AT, has, lane);
            unit_mma<U, ACT, NT>(u, x, x1, has1, nt, kleft, lane, acc);
            x0 += U::SPAN;
            x1 += U::SPAN;
            kleft -= U::SPAN;
        }
        left -= stop - begin;
        if (U::ROW_SCALE) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[m][t][q] *= f[m][q >> 1];
        }
        if (begin == 0 && stop == nk) {
            finish(acc, ti, i);
        } else {
            float4* dst = cut + (warp * 2 + (begin == 0)) * MT * NT * 32 + lane;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < nt)
                        dst[(m * NT + t) * 32] = make_float4(acc[m][t][0], acc[m][t][1], acc[m][t][2], acc[m][t][3]);
        }
        ks = 0;
        next_item(ti, i);
    }
    __syncthreads();
    // The items cut between warps: the first warp that starts inside an item adds
    // its parts in warp order, from the warp before (where the item begins) on.
    if (warp == 0 || u0 >= units || ks0 == 0 || first_unit(warp - 1) > q0 * nk) return;
    const int q_end = (q0 + 1) * nk;
    locate(q0, ti, i);
    const int nt = NT > 1 && s.start[ti + 1] - s.start[ti] > 8 ? 2 : 1;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t][0] = acc[m][t][1] = acc[m][t][2] = acc[m][t][3] = 0.0f;
    for (int w = warp - 1; w < W; ++w) {
        const int from = first_unit(w), to = first_unit(w + 1);
        if (from >= q_end) break;
        if (from == to) continue;
        const float4* part = cut + (w * 2 + (w < warp)) * MT * NT * 32 + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < nt) {
                    const float4 v = part[(m * NT + t) * 32];
                    acc[m][t][0] += v.x;
                    acc[m][t][1] += v.y;
                    acc[m][t][2] += v.z;
                    acc[m][t][3] += v.w;
                }
    }
    finish(acc, ti, i);
}

// ---- down ---------------------------------------------------------------------------

// The end of a tile of up to 32 columns: adds the warps' sums in warp order
// (clearing them for the next tile, if there is one), then the cluster's CTAs',
// in rank order, an equal part of the tile each, and writes it.
template <int ACT, int W>
__device__ __noinline__ void few_tile_end(float* sums, float* both, uint16_t* out, int T, int H, int n0, int n1,
                                          uint32_t rank, int lg, bool last) {
    __syncthreads();
    for (int i = threadIdx.x; i < T * 32; i += W * 32) {
        float* at = sums + (i >> 5) * kFewCols + (i & 31);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += at[w * T * kFewCols];
        both[i] = v;
        if (!last)
            for (int w = 0; w < W; ++w) at[w * T * kFewCols] = 0.0f;
    }
    cluster_sync_all();
    const int part = T * 32 >> lg, end = (rank + 1) * part;
    for (int i = rank * part + threadIdx.x; i < end; i += W * 32) {
        const uint32_t at = smem_u32(both + i);
        float v = ld_dsmem_f32(mapa_shared(at, 0)) + ld_dsmem_f32(mapa_shared(at, 1));
        if (lg > 1) {
            float f[kFewMaxCluster];
#pragma unroll
            for (int r = 2; r < kFewMaxCluster; ++r) f[r] = r >> lg ? 0.0f : ld_dsmem_f32(mapa_shared(at, r));
#pragma unroll
            for (int r = 2; r < kFewMaxCluster; ++r)
                if (!(r >> lg)) v += f[r];
        }
        if (n0 + (i & 31) < n1)
            reinterpret_cast<typename Act<ACT>::T*>(out)[static_cast<size_t>(i >> 5) * H + n0 + (i & 31)] =
                Act<ACT>::from_f(v);
    }
    cluster_sync_all();  // no CTA reuses `both` or leaves while another reads it
}

template <int FMT, int ACT, int NT>
__global__ void __launch_bounds__(FewShape<FMT, NT>::WARPS * 32, FewShape<FMT, NT>::RESIDENT)
few_down_kernel(const FewParams p, const int lg) {  // clusters of 1 << lg CTAs
    using U = Unit<FMT, ACT, false>;
    using S = Stage<U>;
    constexpr int RING = FewShape<FMT, NT>::DN_RING, W = FewShape<FMT, NT>::WARPS, MT = U::MT;
    static_assert(U::ROWS == 32, "32 columns a tile");
    extern __shared__ uint8_t few_smem[];
    float* sums = reinterpret_cast<float*>(few_smem + W * RING * S::BYTES);  // [W][T][kFewCols]
    float* both = sums + W * p.T * kFewCols;                                 // [T][32]: this CTA's sums of a tile
    __shared__ FewPlan s;
    const uint32_t rank = cluster_ctarank();
    // before the wait: only what was complete before the gate/up kernel started
    // (logits, or ids given as inputs) and the weights
    build_plan<W, 8 * NT>(s, p, p.logits != nullptr, false);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int K = p.I, n = s.n;
    int n0, n1;
    part_of(p.H / U::ALIGN, gridDim.x >> lg, blockIdx.x >> lg, n0, n1);
    n0 *= U::ALIGN;
    n1 *= U::ALIGN;
    const int ntiles = (n1 - n0 + 31) / 32;
    const int nks = (K + U::SPAN - 1) / U::SPAN;
    float* mine = sums + warp * p.T * kFewCols;
    for (int i = tid; i < W * p.T * kFewCols; i += W * 32) sums[i] = 0.0f;

    // A tile's units (entry, contraction step), shared by the cluster's warps: this warp's share is the same in every tile
    int u0, u1;
    part_of(n * nks, W << lg, static_cast<int>(rank) * W + warp, u0, u1);
    const int count = u1 - u0;
    const int ti_first = u0 / nks, ks_first = u0 - ti_first * nks;
    uint8_t* ring = few_smem + warp * RING * S::BYTES;

    // The copies: where they are, units left in the tile's share and of the
    // entry, contraction indices to its end
    struct Pos {
        int tile, ti, k, left, of_entry, kleft;
    };
    const Pos start{count > 0 ? 0 : ntiles, ti_first, ks_first * U::SPAN, count, 0, 0};
    Pos l = start;
    typename U::Src src;
    const uint16_t* lx = nullptr;
    bool l_has = false;
    // moves on by a unit; true where a new entry begins
    auto enter = [&](Pos& q) {
        if (q.of_entry > 0) return false;
        q.kleft = K - q.k;
        q.of_entry = (q.kleft + U::SPAN - 1) / U::SPAN;
        return true;
    };
    auto advance = [&](Pos& q) {
        q.kleft -= U::SPAN;
        if (--q.of_entry == 0) {
            q.k = 0;
            ++q.ti;
        }
        if (--q.left == 0) {
            q.left = count;
            q.ti = ti_first;
            q.k = ks_first * U::SPAN;
            q.of_entry = 0;
            ++q.tile;
        }
    };
    auto fetch_w = [&](uint8_t* st, Pos& q) {
        if (enter(q)) {
            const WBase b = expert_base<FMT>(p.down.w, p.down.scales, p.down.zeros, p.H, K, p.down.group_size, s.te[q.ti]);
            const int a = n0 + 32 * q.tile;
            src.aim(b, a, n1 - a, a + 8, n1 - a - 8, q.k, lane);
        }
        if (q.kleft >= U::SPAN) src.load(st, lane);
        else src.load_tail(st, q.kleft, lane);
        src.step();
    };
    auto fetch_h = [&](uint8_t* st, int ti, int kleft, bool entered) {
        if (entered) {
            const int slot = s.start[ti] + g;
            l_has = slot < s.start[ti + 1];
            if (l_has) lx = p.h + static_cast<size_t>(slot) * K + (K - kleft) + U::k_of(0, c);
        }
        Tokens<U>::copy(st + S::X_AT, lx, l_has, kleft, lane);
        lx += U::SPAN;
    };
    for (int d = 0; d < RING - 1 && l.tile < ntiles; ++d) {
        fetch_w(ring + d * S::BYTES, l);
        advance(l);
    }
    pdl_wait();  // h and the routing outputs are complete
    slot_weights<W>(s, p);
    {
        Pos q = start;
        for (int d = 0; d < RING - 1; ++d) {
            if (U::X_RING && q.tile < ntiles) {
                const bool entered = enter(q);
                fetch_h(ring + d * S::BYTES, q.ti, q.kleft, entered);
                advance(q);
            }
            cp_async_commit();
        }
    }
    __syncthreads();  // the slots' weights, and the sums are zero

    float acc[MT][NT][4];
    int stage = 0;
    for (int tile = 0; tile < ntiles; ++tile) {
        const int a = n0 + 32 * tile;
        int left = count, ti = ti_first, ks = ks_first;
        while (left > 0) {  // one entry's units
            const int s0 = s.start[ti], ns = s.start[ti + 1] - s0, nt = NT > 1 && ns > 8 ? 2 : 1, e = s.te[ti];
            const int stop = min(nks, ks + left);
            left -= stop - ks;
            const bool has = g < ns, has1 = NT > 1 && 8 + g < ns;
            const uint16_t* x0 = p.h + static_cast<size_t>(s0 + (has ? g : 0)) * K + ks * U::SPAN + U::k_of(0, c);
            const uint16_t* x1 = has1 ? x0 + static_cast<size_t>(8) * K : x0;
            Tokens<U> x;
            x.clear();
            float f[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                f[m][0] = f[m][1] = U::SCALE_UP;
                if (U::ROW_SCALE) {
                    const float* sc = static_cast<const float*>(p.down.scales) + static_cast<size_t>(p.H) * e + a;
                    f[m][0] = a + U::row_a(m, g) < n1 ? __ldg(sc + U::row_a(m, g)) : 0.0f;
                    f[m][1] = a + U::row_b(m, g) < n1 ? __ldg(sc + U::row_b(m, g)) : 0.0f;
                }
                if (FMT == MOE_W_NVFP4) f[m][0] = f[m][1] = U::SCALE_UP * __ldg(p.down.scale2 + e);
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[m][t][0] = acc[m][t][1] = acc[m][t][2] = acc[m][t][3] = 0.0f;
            }
            int kleft = K - ks * U::SPAN;
            for (; ks < stop; ++ks) {
                if (!U::X_RING) x.fetch(x0, has, kleft, lane);
                __syncwarp();  // every lane is done with the stage refilled now
                if (l.tile < ntiles) {
                    uint8_t* st = ring + (stage == 0 ? RING - 1 : stage - 1) * S::BYTES;
                    const bool entered = l.of_entry == 0;
                    fetch_w(st, l);
                    if (U::X_RING) fetch_h(st, l.ti, l.kleft, entered);
                    advance(l);
                }
                cp_async_commit();
                cp_async_wait_group<RING - 1>();
                __syncwarp();  // scales were copied by other lanes
                const uint8_t* st = ring + stage * S::BYTES;
                if (++stage == RING) stage = 0;
                U u;
                u.open(st, a, a + 8, lane);
                if (U::X_RING) x.open(st + S::X_AT, has, lane);
                unit_mma<U, ACT, NT>(u, x, x1, has1, nt, kleft, lane, acc);
                x0 += U::SPAN;
                x1 += U::SPAN;
                kleft -= U::SPAN;
            }
            // leave the entry: add its products, times the weights, to the tokens' sums
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t > 0 && nt <= t) break;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int slot = 8 * t + 2 * c + q;
                    if (slot < ns) {
                        float* dst = mine + s.slot_tok[s0 + slot] * kFewCols;
                        const float w = s.slot_w[s0 + slot];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            float &da = dst[U::row_a(m, g)], &db = dst[U::row_b(m, g)];
                            da = fmaf(w, f[m][0] * acc[m][t][q], da);
                            db = fmaf(w, f[m][1] * acc[m][t][2 + q], db);
                        }
                    }
                }
            }
            __syncwarp();  // another lane adds to the same token's sums for the next entry
            ks = 0;
            ++ti;
        }
        few_tile_end<ACT, W>(sums, both, p.out, p.T, p.H, a, n1, rank, lg, tile == ntiles - 1);
    }
}

template <int FMT, int ACT, int NT>
cudaError_t launch_few_nt(const FewParams& p, int sms, cudaStream_t st) {
    using F = FewShape<FMT, NT>;
    using GU = Unit<FMT, ACT, true>;
    using DN = Unit<FMT, ACT, false>;
    constexpr int gu_smem =
        F::WARPS * (F::GU_RING * Stage<GU>::BYTES + static_cast<int>(sizeof(float4)) * 2 * GU::MT * NT * 32);
    constexpr int dn_ring = F::WARPS * F::DN_RING * Stage<DN>::BYTES;
    constexpr int dn_token = static_cast<int>(sizeof(float)) * (F::WARPS * kFewCols + 32);
    constexpr int dn_most = dn_ring + dn_token * MOE_MAX_FEW_TOKENS;
    static_assert(gu_smem + sizeof(FewPlan) <= 232448 && dn_most + sizeof(FewPlan) <= 232448, "shared memory");
    static int configured_for = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        if (set_smem_limit(reinterpret_cast<const void*>(few_gate_up_kernel<FMT, ACT, NT>), gu_smem) != MOE_OK ||
            set_smem_limit(reinterpret_cast<const void*>(few_down_kernel<FMT, ACT, NT>), dn_most) != MOE_OK)
            return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(F::WARPS * 32);
    cfg.attrs = attr;
    static int most[kFewMaxLg + 1];  // by lg: clusters that fit the GPU at once, a CTA per SM
    if (configured_for != dev) {
        cfg.dynamicSmemBytes = dn_most;
        cfg.numAttrs = 1;
        for (int lg = 1; lg <= kFewMaxLg; ++lg) {
            attr[0].val.clusterDim.x = 1 << lg;
            cfg.gridDim = dim3(1 << lg);
            if (cudaOccupancyMaxActiveClusters(&most[lg], few_down_kernel<FMT, ACT, NT>, &cfg) != cudaSuccess)
                return cudaGetLastError();
            most[lg] = most[lg] < sms >> lg ? most[lg] : sms >> lg;
        }
        configured_for = dev;
    }
    // The cluster's size: the fewest units a warp. A tile's end counts as four (about 1.5 us)
    const int cols = p.H / DN::ALIGN;
    const int units = (p.T * p.k < p.E ? p.T * p.k : p.E) * ((p.I + DN::SPAN - 1) / DN::SPAN);
    int best = 1, groups = 1;
    int64_t least = INT64_MAX;
    for (int lg = 1; lg <= kFewMaxLg; ++lg) {
        const int n = most[lg] < cols ? most[lg] : cols, warps = F::WARPS << lg;
        if (n < 1) break;
        const int tiles = ((cols + n - 1) / n * DN::ALIGN + 31) / 32;
        const int64_t steps = static_cast<int64_t>(tiles) * ((units + warps - 1) / warps + 4);
        if (steps < least) {
            least = steps;
            best = lg;
            groups = n;
        }
    }
    const cudaError_t e = launch_pdl(few_gate_up_kernel<FMT, ACT, NT>, sms, (F::WARPS + 1) * 32, gu_smem, st, p);
    if (e != cudaSuccess) return e;
    attr[0].val.clusterDim.x = 1 << best;
    cfg.gridDim = dim3(groups << best);
    cfg.dynamicSmemBytes = dn_ring + dn_token * p.T;
    cfg.stream = st;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_down_kernel<FMT, ACT, NT>, p, best);
}

// Token tiles of 8 a product takes: one, and an expert with more tokens is read
// again (mostly from L2), or two, where most experts have more than 6. us at one
// / two, H = 2048, T = 32, k = 8, E = 48 and 32: NVFP4 70 / 73 and 64 / 58, FP8
// 64 / 69 and 57 / 55, GPTQ 70 / 76 and 64.4 / 63.7. Two never paid for bf16 (90 /
// 111 at E = 32, 78 / 90 at E = 16).
template <int FMT, int ACT>
cudaError_t launch_few(const FewParams& p, int sms, cudaStream_t st) {
    if constexpr (FMT != MOE_W_BF16)
        if (p.T > 8 && p.T * p.k > 6 * p.E) return launch_few_nt<FMT, ACT, 2>(p, sms, st);
    return launch_few_nt<FMT, ACT, 1>(p, sms, st);
}

}  // namespace moe
