// Ragged products on the 5th-generation tensor cores, on CTA pairs
// (tcgen05.mma.cta_group::2, M = 256).
//
// Rows form (the product, and the gradient of its input):
//     out[r, j] = sum_c a[r, c] W_e[j, c]            rows r of group e
//   The weights are the MMA's M operand (256 output columns a tile, 128 per CTA), up to
//   256 rows of one group its N operand (half of them per CTA). So a group of few rows
//   costs little more than its weights' bytes, and rows need no padding: N is the tile's
//   height in steps of 16, the epilogue stores the rows that there are. For the input's
//   gradient the contraction runs over the weight's slow index: the same bytes, with
//   64 x 64 boxes laid down as they lie and read as an MN-major operand, so that no
//   transposed copy of the weights is needed.
// Gradient form (the weight's gradient):
//     dw_e[n, k] = sum_{r in e} dy[r, n] x[r, k]
//   Both operands are MN-major, the contraction runs over the group's rows, 64 a block.
//   A group's last block takes as many MMAs as it has units of 16 rows; the rows of its
//   last unit that belong to the next group (or to nobody: they may hold infinities) are
//   set to zeros in shared memory, in both operands, by a warp of each CTA, before the
//   MMA may read them.
//
// Roles: warps 0 and 6 copy the two operands (TMA, 128-byte swizzle; a thread takes 90
// to 190 clocks per copy, and there are up to four a block), warp 1 of the even CTA (the
// leader) issues the MMAs, warps 2 to 5 are the epilogue, warp 7 clears tails. Two
// accumulators of 256 TMEM columns let the epilogue of a tile run beside the next one's
// MMAs. Every wait is bounded.
//
// Few tiles with a long contraction: a cluster of PARTS pairs takes one tile, each pair a
// part of the contraction, and each CTA adds a slice of the tile's rows from all parts in
// their order (distributed shared memory).
#pragma once

#include "ragged.cuh"

namespace moe {
namespace ragged {
// (in a namespace of its own file: every .cu that includes this has its own kernels)
namespace {

enum { ROWS_FWD = 0, ROWS_BACK = 1, WGRAD = 2 };

constexpr int BK = 64;
constexpr int STAGES = 6;
constexpr int OPER = 128 * BK * 2;  // bytes of a CTA's share of an operand per stage
constexpr int STAGE = 2 * OPER;
constexpr int THREADS = 256;
constexpr int SG = 36;                    // row stride (floats) of a warp's staging area: 16-byte reads without conflicts
constexpr int STG_WARP = 32 * SG * 4;     // rows form: 32 rows x 32 columns f32; gradient form: 32 x 128 bytes
constexpr int STG_AT = STAGES * STAGE;

struct Tail {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t tloc[STAGES], tready[STAGES];  // gradient form: a tail block's copies of this CTA, and both CTAs' cleared tails
    uint64_t tfull[2], tempty[2], mma_done;
    uint32_t tmem_base;
    int abort_flag, n_tiles, jt;
    int off[MOE_MAX_EXPERTS + 1];
    int tstart[MOE_MAX_EXPERTS + 1];
};
constexpr int TAIL_AT = STG_AT + 4 * STG_WARP;
constexpr int SMEM = 1024 + TAIL_AT + (static_cast<int>(sizeof(Tail)) + 127) / 128 * 128;
static_assert(SMEM <= 232448, "shared memory over the limit");
static_assert(STG_AT % 1024 == 0, "the gradient form's staging areas are 1024-byte swizzle atoms");

// ---- operands -------------------------------------------------------------------------
// MN-major operand with the 128-byte swizzle, as a TMA box of 64 elements (128 bytes) x 64
// contraction indices lays it down: 8 contraction indices are 1024 bytes (the stride
// offset), the next 64 elements are 8192 bytes on (the leading offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(8192u >> 4) << 16 |
           static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;  // instruction descriptor: operand is MN-major

// 3-D load of a CTA pair, to a barrier of the cluster
__device__ __forceinline__ void load_3d_pair(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// mbar_wait, with an acquire of what the other CTA released to it
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
    if (!mbar_wait(bar, parity, w)) return false;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return true;
}

// ---- tiles ------------------------------------------------------------------------------
struct Tile {
    int e;
    int j0;        // rows form: first output column; gradient form: first n
    int m0, rows;  // rows form: first row and rows of the tile; gradient form: the group's
    int n;         // the MMA's N
    int k0;        // gradient form: first k
};

// Rows form: a group's rows are cut into tiles of nearly equal height, in units of 16 rows
// and at most maxu of them. Every CTA builds the list from the offsets: the tiles of group
// e begin at tstart[e], its row tiles fastest, then output columns. Returns whether the
// offsets are bad (no tile then).
template <int MODE>
__device__ __forceinline__ int build_tiles(Tail& s, const RaggedParams& p) {
    const int tid = threadIdx.x, lane = tid & 31, E = p.E;
    for (int i = tid; i <= E; i += THREADS) s.off[i] = p.offsets ? p.offsets[i] : (i ? p.rows : 0);
    const int jt = (p.J + 255) / 256;
    if (tid == 0) {
        s.abort_flag = 0;
        s.jt = jt;
    }
    __syncthreads();
    int bad = 0;
    for (int i = tid; i < E; i += THREADS) bad |= s.off[i + 1] < s.off[i];
    if (tid == 0) bad |= s.off[0] < 0 || s.off[E] > p.rows;
    bad = __syncthreads_or(bad);
    if (MODE == WGRAD) {
        if (tid == 0) s.n_tiles = bad ? 0 : E * jt * ((p.C + p.maxu - 1) / p.maxu);
        return bad;
    }
    if (tid < 32) {
        auto tiles = [&](int e) {
            return e < E && !bad ? ((s.off[e + 1] - s.off[e] + 15) / 16 + p.maxu - 1) / p.maxu * jt : 0;
        };
        const int per = (E + 31) / 32;
        int loc = 0;
        for (int j = 0; j < per; ++j) loc += tiles(lane * per + j);
        int inc = loc;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        int run = inc - loc;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            if (e < E) s.tstart[e] = run;
            run += tiles(e);
        }
        if (lane == 31) s.n_tiles = inc;
    }
    return bad;
}

template <int MODE> __device__ __forceinline__ Tile get_tile(const Tail& s, const RaggedParams& p, int tile) {
    Tile t;
    if (MODE == WGRAD) {
        const int kt = (p.C + p.maxu - 1) / p.maxu, per = s.jt * kt;
        t.e = tile / per;
        const int in = tile - t.e * per, jn = in / kt;
        t.j0 = jn * 256;
        t.k0 = (in - jn * kt) * p.maxu;
        t.m0 = s.off[t.e];
        t.rows = s.off[t.e + 1] - t.m0;
        t.n = p.maxu;
        return t;
    }
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.tstart[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    // (of groups that begin at the same tile all but the last are empty)
    t.e = lo;
    const int v = s.off[lo + 1] - s.off[lo], U = (v + 15) / 16, mt = (U + p.maxu - 1) / p.maxu;
    const int local = tile - s.tstart[lo], jn = local / mt, i = local - jn * mt;
    const int u0 = static_cast<int>(static_cast<int64_t>(U) * i / mt),
              u1 = static_cast<int>(static_cast<int64_t>(U) * (i + 1) / mt);
    t.m0 = s.off[lo] + 16 * u0;
    t.rows = min(v, 16 * u1) - 16 * u0;
    t.n = 16 * (u1 - u0);
    t.j0 = jn * 256;
    t.k0 = 0;
    return t;
}

// ---- epilogues --------------------------------------------------------------------------

// Rows form: up to 32 rows x 32 columns z (lane = column, v[i] = row m + i) of a warp to
// memory, through its staging area so that they leave as 16-byte pieces of 8 columns; the
// piece's activation function and residual are applied on the way, in f32.
template <int ACT>
__device__ __forceinline__ void store_rows(const RaggedParams& p, const float (&v)[32], float* stg, int lane, int m,
                                           int rows, int col0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) stg[i * SG + lane] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (i * 32 + lane) >> 2, col = col0 + 8 * (lane & 3);
        if (r >= rows || col >= p.J) continue;
        const float4 lo = *reinterpret_cast<const float4*>(stg + r * SG + 8 * (lane & 3));
        const float4 hi = *reinterpret_cast<const float4*>(stg + r * SG + 8 * (lane & 3) + 4);
        float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const size_t at = static_cast<size_t>(m + r) * p.J + col;
        if (p.pre) *reinterpret_cast<uint4*>(p.pre + at) = pack8<ACT>(f);
        if (p.fn != MOE_FN_NONE)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fn_value(p.fn, f[j]);
        if (p.residual) {
            float g[8];
            unpack8<ACT>(*reinterpret_cast<const uint4*>(p.residual + at), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = pack8<ACT>(f);
    }
    __syncwarp();
}

template <int ACT>
__device__ __forceinline__ float bias_of(const RaggedParams& p, int col) {
    if (!p.bias || col >= p.J) return 0.0f;
    return Act<ACT>::to_f(reinterpret_cast<const typename Act<ACT>::T*>(p.bias)[col]);
}

template <int ACT>
__device__ __forceinline__ void rows_epilogue(const RaggedParams& p, uint32_t ta, float* stg, const Tile& t, int col0,
                                              int lane) {
    const float b = bias_of<ACT>(p, col0 + lane);
    uint32_t nx[32];
    tmem_ld32(ta, nx);
#pragma unroll 1
    for (int c = 0; c < t.rows; c += 32) {
        float v[32];
        tmem_ld_wait_regs(nx);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(nx[j]) + b;
        if (c + 32 < t.rows) tmem_ld32(ta + c + 32, nx);  // in flight while this one is stored
        store_rows<ACT>(p, v, stg, lane, t.m0 + c, t.rows - c, col0);
    }
}

// A tensor core's f32 sums are cut, not rounded, to 24 bits at each step of 16 products:
// where sums grow steadily, 30000 rows in one accumulator left them 4e-5 short. An f32
// gradient therefore takes its rows in chunks of 4096 (5e-6), one accumulator each, and
// the epilogue adds the chunks in f32, through dw itself. (16-bit gradients are rounded
// to 2^-9 or 2^-12 anyway and take one.)
constexpr int CHUNK = 64;  // blocks

__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Gradient form: lane = row n of dw, columns k. 128 bytes of a row (32 f32 or 64 16-bit
// values) go to the staging area, 16-byte pieces swizzled by row, and leave by a TMA store,
// which leaves out what lies past the weight's edges.
template <int ACT, bool F32>
__device__ __forceinline__ void wgrad_epilogue(const RaggedParams& p, const CUtensorMap* tm_out, uint32_t ta, uint8_t* stg,
                                               const Tile& t, int n0, int lane, bool first, bool last) {
    constexpr int COLS = F32 ? 32 : 64;
    const int n = n0 + lane;
    const bool row = n < p.J;
    const size_t at = (static_cast<size_t>(t.e) * p.J + (row ? n : 0)) * p.C;
    // what is added: later chunks find there what this thread stored itself
    const float* add = first ? (p.addend ? p.addend + at : nullptr) : static_cast<const float*>(p.out) + at;
#pragma unroll 1
    for (int c = 0; c < p.maxu && t.k0 + c < p.C; c += COLS) {
        uint4 piece[8];
#pragma unroll
        for (int h = 0; h < COLS; h += 32) {
            uint32_t u[32];
            float v[32];
            if (t.rows > 0) {
                tmem_ld32(ta + c + h, u);
                if (F32 && add && row) {  // the loads run beside each other
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (t.k0 + c + 4 * q < p.C)
                            piece[q] = *reinterpret_cast<const uint4*>(add + t.k0 + c + 4 * q);
                }
                tmem_ld_wait_regs(u);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
                if (F32 && add && row) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (t.k0 + c + 4 * q < p.C) {
                            v[4 * q] += __uint_as_float(piece[q].x);
                            v[4 * q + 1] += __uint_as_float(piece[q].y);
                            v[4 * q + 2] += __uint_as_float(piece[q].z);
                            v[4 * q + 3] += __uint_as_float(piece[q].w);
                        }
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (F32 && add && row && t.k0 + c + 4 * q < p.C)
                        f = *reinterpret_cast<const float4*>(add + t.k0 + c + 4 * q);
                    v[4 * q] = f.x;
                    v[4 * q + 1] = f.y;
                    v[4 * q + 2] = f.z;
                    v[4 * q + 3] = f.w;
                }
            }
            if (F32) {
                if (!last) {
                    float* own = static_cast<float*>(p.out) + at + t.k0 + c;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (row && t.k0 + c + 4 * q < p.C)
                            *reinterpret_cast<float4*>(own + 4 * q) =
                                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    continue;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    piece[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                          __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    piece[h / 8 + q] = make_uint4(Act<ACT>::pack2(v[8 * q], v[8 * q + 1]),
                                                  Act<ACT>::pack2(v[8 * q + 2], v[8 * q + 3]),
                                                  Act<ACT>::pack2(v[8 * q + 4], v[8 * q + 5]),
                                                  Act<ACT>::pack2(v[8 * q + 6], v[8 * q + 7]));
            }
        }
        if (F32 && !last) continue;
        if (lane == 0) store_wait_read();  // the area's last store
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(stg + lane * 128 + 16 * (q ^ (lane & 7))) = piece[q];
        fence_proxy_async_smem();
        if (F32 && !first) fence_proxy_async_global();  // the store overwrites this thread's earlier ones
        __syncwarp();
        if (lane == 0 && n0 < p.J) {
            store_3d(tm_out, stg, t.k0 + c, n0, t.e);
            store_commit();
        }
    }
}

// ---- the kernel ---------------------------------------------------------------------------
// tm_a: the M operand (weights; dy), tm_b: the N operand (rows; x), tm_out: the gradient.
template <int MODE, int ACT, bool F32, int PARTS>
__global__ void __launch_bounds__(THREADS, 1)
ragged_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_out, const RaggedParams p) {
    static_assert(PARTS == 1 || MODE != WGRAD, "only the rows form is split");
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    Tail& s = *reinterpret_cast<Tail*>(smem + TAIL_AT);
    const WaitCtx wc{&s.abort_flag, p.err, p.wait_ns};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
    const int part = static_cast<int>(crank >> 1);
    const int first = blockIdx.x / (2 * PARTS), step = gridDim.x / (2 * PARTS);

    const int bad = build_tiles<MODE>(s, p);  // identical in every CTA
    if (tid == 0) {
        if (bad && blockIdx.x == 0) set_err(p.err, MOE_DEV_ERR_OFFSETS);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.tloc[i], 1);
            mbar_init(&s.tready[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 8);  // the pair's epilogue warps
        }
        mbar_init(&s.mma_done, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const int n_tiles = s.n_tiles;
    if (first >= n_tiles) return;  // the same in all CTAs of the cluster: nothing allocated yet

    if (warp == 1) {
        tmem_alloc_pair(&s.tmem_base, 512);
        tmem_relinquish_pair();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        if (MODE == WGRAD) tma_prefetch_desc(&tm_out);
    }
    tc_fence_before();
    cluster_sync_all();  // barriers initialised, TMEM allocated
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    const uint32_t lead_full = mapa_shared(smem_u32(&s.full[0]), lead);
    const uint32_t lead_tempty = mapa_shared(smem_u32(&s.tempty[0]), lead);
    const uint32_t lead_tready = mapa_shared(smem_u32(&s.tready[0]), lead);
    const int KBall = (p.C + BK - 1) / BK;
    const int kb0 = PARTS > 1 ? KBall * part / PARTS : 0;
    const int kb1 = PARTS > 1 ? KBall * (part + 1) / PARTS : KBall;
    // this CTA's bytes of a stage
    const uint32_t b_bytes = MODE == WGRAD ? p.maxu * 64 : p.maxu * 8 * 128;
    auto blocks_of = [&](const Tile& t) { return MODE == WGRAD ? (t.rows + BK - 1) / BK : kb1 - kb0; };

    if (warp == 0 || warp == 6) {
        if (lane == 0) {
            // ---------------- copies: warp 0 the M operand, warp 6 the N operand ----------------
            const bool is_a = warp == 0;
            uint32_t stage = 0, phase = 0, used = 0, tpar = 0;
            long issued = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                const Tile t = get_tile<MODE>(s, p, tile);
                const int nb = blocks_of(t);
                for (int b = 0; b < nb; ++b) {
                    if (!mbar_wait(&s.empty[stage], phase ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    const bool tail = MODE == WGRAD && b + 1 == nb && t.rows % 16 != 0;
                    uint32_t bar = lead_full + stage * 8;
                    if (tail) {
                        bar = mapa_shared(smem_u32(&s.tloc[stage]), crank);
                        if (is_a) mbar_arrive_expect_tx(&s.tloc[stage], OPER + b_bytes);
                        if (is_a && rank == 0) mbar_arrive(&s.full[stage]);
                        used |= 1u << stage;
                        tpar ^= 1u << stage;  // bit: uses so far, mod 2
                    } else if (is_a && rank == 0) {
                        mbar_arrive_expect_tx(&s.full[stage], 2 * (OPER + b_bytes));
                    }
                    uint8_t* dst = smem + stage * STAGE + (is_a ? 0 : OPER);
                    if (MODE == WGRAD) {
                        const int r = t.m0 + b * BK;
                        if (is_a) {
                            const int n = t.j0 + 128 * static_cast<int>(rank);
                            tma_load_2d_pair(dst, &tm_a, n, r, bar);
                            tma_load_2d_pair(dst + 8192, &tm_a, n + 64, r, bar);
                        } else {
                            const int k = t.k0 + p.maxu / 2 * static_cast<int>(rank);
                            tma_load_2d_pair(dst, &tm_b, k, r, bar);
                            if (p.maxu == 256) tma_load_2d_pair(dst + 8192, &tm_b, k + 64, r, bar);
                        }
                    } else {
                        const int c = (kb0 + b) * BK;
                        if (is_a) {
                            const int j = t.j0 + 128 * static_cast<int>(rank);
                            if (MODE == ROWS_FWD) {
                                load_3d_pair(dst, &tm_a, c, j, t.e, bar);
                            } else {
                                load_3d_pair(dst, &tm_a, j, c, t.e, bar);
                                load_3d_pair(dst + 8192, &tm_a, j + 64, c, t.e, bar);
                            }
                        } else {
                            // (the box has maxu * 8 rows; the MMA reads n / 2 of them)
                            tma_load_2d_pair(dst, &tm_b, c, t.m0 + static_cast<int>(rank) * (t.n / 2), bar);
                        }
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (is_a) {  // let every copy land before either CTA may exit
                if (rank == 0) {
                    const long from = issued > STAGES ? issued - STAGES : 0;
                    for (long j = from; j < issued; ++j)
                        mbar_drain(&s.full[j % STAGES], static_cast<uint32_t>((j / STAGES) & 1), kWaitLimitNs / 8);
                }
                for (int i = 0; i < STAGES; ++i)
                    if (used >> i & 1u) mbar_drain(&s.tloc[i], (tpar >> i & 1u) ^ 1u, kWaitLimitNs / 8);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMAs (leader) ----------------
            const uint32_t major = MODE == WGRAD ? kMajorA | kMajorB : MODE == ROWS_BACK ? kMajorA : 0u;
            constexpr uint32_t STEP_K = 32 >> 4, STEP_MN = 2048 >> 4;  // 16 contraction indices on, in descriptor units
            constexpr uint32_t step_a = MODE == ROWS_FWD ? STEP_K : STEP_MN, step_b = MODE == WGRAD ? STEP_MN : STEP_K;
            uint32_t stage = 0, phase = 0, tpar = 0;
            int local = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                const Tile t = get_tile<MODE>(s, p, tile);
                const int nb = blocks_of(t);
                const uint32_t idesc = f16_idesc(ACT, 256, t.n) | major;
                uint32_t d = 0;
                int acc = 0, b0 = 0;  // the accumulator, and the first block that goes there
                for (int b = 0; b < nb || b == 0; ++b) {
                    if (b == 0 || (F32 && b % CHUNK == 0)) {
                        if (b > 0) tc_commit_pair(&s.tfull[acc], static_cast<uint16_t>(3u << lead));
                        acc = local & 1;
                        const uint32_t aph = (local >> 1) & 1;
                        ++local;
                        if (!mbar_wait(&s.tempty[acc], aph ^ 1, wc)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        d = tmem + acc * 256;
                        b0 = b;
                        if (nb == 0) break;
                    }
                    if (!mbar_wait(&s.full[stage], phase, wc)) {
                        ok = false;
                        break;
                    }
                    int steps = BK / 16;
                    if (MODE == WGRAD && b + 1 == nb) {
                        steps = (t.rows - b * BK + 15) / 16;
                        if (t.rows % 16 != 0) {  // both CTAs have cleared their tails
                            if (!wait_cluster(&s.tready[stage], tpar >> stage & 1u, wc)) {
                                ok = false;
                                break;
                            }
                            tpar ^= 1u << stage;
                        }
                    }
                    tc_fence_after();
                    const uint32_t at = smem_u32(smem + stage * STAGE);
                    const uint64_t ad = MODE == ROWS_FWD ? sw128_desc(at) : mn_desc(at);
                    const uint64_t bd = MODE == WGRAD ? mn_desc(at + OPER) : sw128_desc(at + OPER);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        if (MODE != WGRAD || k < steps)
                            tc_mma_pair(d, ad + k * step_a, bd + k * step_b, idesc, b > b0 || k > 0);
                    tc_commit_pair(&s.empty[stage], static_cast<uint16_t>(3u << lead));
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair(&s.tfull[acc], static_cast<uint16_t>(3u << lead));
            }
            tc_commit_pair(&s.mma_done, static_cast<uint16_t>(1u << lead));
            mbar_drain(&s.mma_done, 0, kWaitLimitNs / 8);
        }
        __syncwarp();
    } else if (warp == 7) {
        if (MODE == WGRAD) {
            // ---------------- tails: rows of a group's last unit of 16 that are not the group's ----------------
            uint32_t stage = 0, tpar = 0;
            for (int tile = first; tile < n_tiles; tile += step) {
                const Tile t = get_tile<MODE>(s, p, tile);
                const int nb = blocks_of(t);
                if (nb == 0) continue;
                const uint32_t last = (stage + nb - 1) % STAGES;
                stage = (stage + nb) % STAGES;
                if (t.rows % 16 == 0) continue;
                if (!mbar_wait_warp(&s.tloc[last], tpar >> last & 1u, wc)) break;
                tpar ^= 1u << last;
                const int r0 = t.rows - (nb - 1) * BK, r1 = (r0 + 15) / 16 * 16;
                // row r of each 64-element group is the 128 bytes at 128 r (the swizzle moves bytes within them)
                uint8_t* base = smem + last * STAGE;
                const int chunks = 16 + p.maxu / 16;  // 16-byte pieces a row has in both operands
                for (int i = lane; i < (r1 - r0) * chunks; i += 32) {
                    const int r = r0 + i / chunks, c = i % chunks;
                    *reinterpret_cast<uint4*>(base + (c >> 3) * 8192 + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead_tready + last * 8);
            }
        }
    } else if (PARTS == 1) {
        // ---------------- epilogue ----------------
        const int q = warp & 3;  // TMEM lane quarter
        uint8_t* stg = smem + STG_AT + (MODE == WGRAD ? (warp - 2) * 4096 : (warp - 2) * STG_WARP);
        int local = 0;
        bool ok = true;
        for (int tile = first; tile < n_tiles && ok; tile += step) {
            const Tile t = get_tile<MODE>(s, p, tile);
            const int chunks = F32 ? max(1, (blocks_of(t) + CHUNK - 1) / CHUNK) : 1;
            for (int ch = 0; ch < chunks; ++ch) {
                const int acc = local & 1;
                const uint32_t aph = (local >> 1) & 1;
                ++local;
                if (!mbar_wait_warp(&s.tfull[acc], aph, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
                const int col0 = t.j0 + 128 * static_cast<int>(rank) + 32 * q;
                if (MODE == WGRAD) wgrad_epilogue<ACT, F32>(p, &tm_out, ta, stg, t, col0, lane, ch == 0, ch + 1 == chunks);
                else rows_epilogue<ACT>(p, ta, reinterpret_cast<float*>(stg), t, col0, lane);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&s.tempty[acc]);
                    else mbar_arrive_cluster(lead_tempty + acc * 8);
                }
            }
        }
        if (MODE == WGRAD && lane == 0) store_wait();
    }

    __syncwarp();
    if (PARTS > 1) {
        // ---------------- a split tile's sums, from all parts ----------------
        const Tile t = get_tile<MODE>(s, p, first);
        const bool epi = warp >= 2 && warp < 6;
        const int q = warp & 3, me = 32 * q + lane;
        bool ok = true;
        if (epi) {
            ok = mbar_wait_warp(&s.tfull[0], 0, wc);
            tc_fence_after();
        }
        __syncwarp();
        cluster_sync_all();  // every pair's MMAs are complete: the stages are free
        float* sums = reinterpret_cast<float*>(smem);  // [source part][row of the slice][128 columns]
        const int per = t.n / PARTS;                   // rows of a slice (n is a multiple of 16)
        if (epi) {
            const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < t.n; c += 32) {
                uint32_t u[32];
                tmem_ld32(ta + c, u);
                tmem_ld_wait_regs(u);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int dst = (c + j) / per;
                    if (c + j < t.n) {
                        const uint32_t to =
                            mapa_shared(smem_u32(sums + (part * per + c + j - dst * per) * 128 + me), 2 * dst + rank);
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(u[j]) : "memory");
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (epi && ok) {
            const int col0 = t.j0 + 128 * static_cast<int>(rank) + 32 * q;
            const float b = bias_of<ACT>(p, col0 + lane);
            float* stg = reinterpret_cast<float*>(smem + STG_AT + (warp - 2) * STG_WARP);
            const int have = min(per, t.rows - part * per);
#pragma unroll 1
            for (int c = 0; c < have; c += 32) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    v[j] = 0.0f;
                    if (c + j < have) {
                        v[j] = sums[(c + j) * 128 + me];
#pragma unroll
                        for (int r = 1; r < PARTS; ++r) v[j] += sums[(r * per + c + j) * 128 + me];
                        v[j] += b;
                    }
                }
                store_rows<ACT>(p, v, stg, lane, t.m0 + part * per + c, have - c, col0);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the leader's MMAs read the peer's shared memory and write its TMEM
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---- launch -----------------------------------------------------------------------------

// clusters of 2 PARTS CTAs that the current device runs at once
template <typename Kernel> int prepare(Kernel kernel, int parts, int& clusters, const char* who) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    const int sms = sm_count();
    cfg.gridDim = dim3(sms > 0 ? sms / (2 * parts) * (2 * parts) : 2 * parts);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int rc = set_smem_limit(reinterpret_cast<const void*>(kernel), SMEM);
    if (rc != MOE_OK) return rc;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess || clusters <= 0)
        return fail(MOE_ERR_CUDA, "%s: cannot place clusters of %d CTAs: %s", who, 2 * parts, cudaGetErrorString(e));
    return MOE_OK;
}

template <int MODE, int ACT, bool F32, int PARTS>
int launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, const RaggedParams& p, int64_t tiles,
           cudaStream_t st, const char* who) {
    auto kernel = ragged_kernel<MODE, ACT, F32, PARTS>;
    static int configured_for = -1, clusters = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        int n = 0;
        const int rc = prepare(kernel, PARTS, n, who);
        if (rc != MOE_OK) return rc;
        clusters = n;
        configured_for = dev;
    }
    if (tiles > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
    if (tiles <= 0) return MOE_OK;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * PARTS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    // a split tile is one cluster's; otherwise clusters walk the tiles
    cfg.gridDim = dim3(static_cast<unsigned>(2 * PARTS * (PARTS > 1 || tiles < clusters ? tiles : clusters)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, b, out, p);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

// Rows form: tile height and split.
template <int ACT, int MODE> int rows_form(const RaggedArgs& g) {
    RaggedParams p = g.p;
    // rows a group has, if all have the same
    const int64_t each = (static_cast<int64_t>(p.rows) + p.E - 1) / p.E;
    const int units = static_cast<int>((each + 15) / 16 < 16 ? (each + 15) / 16 : 16);
    p.maxu = 1;
    while (p.maxu < units) p.maxu *= 2;
    int parts = 1;
    const int64_t jt = (p.J + 255) / 256;
    if (p.E == 1) {
        const int64_t tiles = ((p.rows + 15) / 16 + p.maxu - 1) / p.maxu * jt;
        const int kb = (p.C + BK - 1) / BK;
        while (parts < 4 && tiles * parts * 2 <= 72 && kb >= 8 * parts) parts *= 2;
    }
    CUtensorMap a, b;
    int rc = make_tmap_3d(&a, const_cast<void*>(g.w), g.act, g.K, g.N, p.E, 64, MODE == ROWS_FWD ? 128 : 64);
    if (rc == MOE_OK) rc = make_tmap_2d(&b, g.a, p.rows, p.C, p.maxu * 8, g.act);
    if (rc != MOE_OK) return rc;
    // row tiles at most: one more per group than the rows fill
    const int64_t tiles = ((p.rows + 16 * p.maxu - 1) / (16 * p.maxu) + (p.E > 1 ? p.E : 0)) * jt;
    switch (parts) {
        case 1: return launch<MODE, ACT, false, 1>(a, b, b, p, tiles, g.st, g.who);
        case 2: return launch<MODE, ACT, false, 2>(a, b, b, p, tiles, g.st, g.who);
        default: return launch<MODE, ACT, false, 4>(a, b, b, p, tiles, g.st, g.who);
    }
}

}  // namespace
}  // namespace ragged
}  // namespace moe
