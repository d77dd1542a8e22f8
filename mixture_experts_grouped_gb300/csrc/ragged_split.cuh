// Products of few tiles: one 128-column tile to a cluster of CTAs, each with a part of the
// contraction.
//
// With few rows a product is bound by its weights' bytes, and only if every SM streams
// them: 4096 columns are 16 tiles of the pair form, and 32 SMs drew 2.3 TB/s. Here a tile is
// 128 output columns (the MMA's M operand, one CTA) by up to 128 rows (its N operand), and
// up to 8 CTAs share its contraction, two CTAs to an SM. Each then adds a slice of the
// tile's rows from all parts, in their order, through distributed shared memory, and
// finishes it. (Clusters of pairs do not fit as well: of 8 CTAs with an SM each, 15 are
// placed at once.) Every wait is bounded. Measured: 37 x 4096 x 14336 26.5 us, 4.5 TB/s (52
// with pairs); 37 x 2816 x 2048 8.0 us, most of it launch, first copies, and the cluster's two
// meetings (2.5 us).
//
// Groups (with offsets, at most 128 rows in all): a tile for every group and 128 columns;
// those of empty groups leave at once.
//
// Gradient of one group's weight: a tile is 128 rows n by 128 columns k of it, the
// contraction runs over the rows (past their end the copies bring zeros).
#pragma once

#include "ragged_tc.cuh"

namespace moe {
namespace ragged {
namespace {

constexpr int SPLIT_THREADS = 192;
constexpr int SPLIT_MAX_STAGES = 8;
constexpr int SPLIT_ROWS = 128;  // most rows of a tile
static_assert(SPLIT_MAX_ROWS <= SPLIT_ROWS, "a group is one tile");
constexpr int SPLIT_PARTS = 8;   // most CTAs of a tile

constexpr int STG_ROWS = 16;  // rows of an epilogue warp's staging area
constexpr int SG = 36;        // and their stride (floats): 16-byte reads without conflicts

struct SplitTail {
    uint64_t full[SPLIT_MAX_STAGES], empty[SPLIT_MAX_STAGES], done;
    uint64_t sums[2], taken[2];  // a chunk's sums there, and read
    uint32_t tmem_base;
    int abort_flag;
};

struct SplitParams {
    RaggedParams r;
    int parts, stages;
    int mt;        // row tiles of one group; gradient: tiles of k
    int box;       // rows of the N operand's boxes: the tallest tile, or with groups 16, as many boxes as a tile needs
    int stage;     // bytes of a stage
    int tmem;      // TMEM columns
    int tail_at;   // after the stages
};

__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    tma_load_3d(dst, map, c0, c1, c2, bar);
}

struct Residual {
    uint4 v[2];
    __device__ __forceinline__ void load(const RaggedParams& p, int lane, int m, int rows, int col0) {
        if (!p.residual) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Piece c(i, lane, col0);
            if (c.in(p, rows)) v[i] = *reinterpret_cast<const uint4*>(p.residual + c.at(p, m));
        }
    }
};

// Up to 16 rows x 32 columns z (lane = column, v[i] = row m + i) of a warp to
// memory, through its staging area so that they leave as pieces; the piece's activation
// function and residual are applied on the way, in f32.
template <int ACT, int KIND>
__device__ __forceinline__ void store_rows(const RaggedParams& p, const float (&v)[16], const Residual& res, float* stg,
                                           int lane, int m, int rows, int col0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) stg[i * SG + lane] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Piece c(i, lane, col0);
        if (!c.in(p, rows)) continue;
        const float4 lo = *reinterpret_cast<const float4*>(stg + c.r * SG + 8 * (lane & 3));
        const float4 hi = *reinterpret_cast<const float4*>(stg + c.r * SG + 8 * (lane & 3) + 4);
        float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const size_t at = c.at(p, m);
        if (KIND == FULL) {
            if (p.pre) *reinterpret_cast<uint4*>(p.pre + at) = pack8<ACT>(f);
            fn_values(p.fn, f);
            if (p.residual) {
                float g[8];
                unpack8<ACT>(res.v[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += g[j];
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = pack8<ACT>(f);
    }
    __syncwarp();
}

// Addends of 16 columns k .. of row n of one group's weight gradient, of those there are. (All at once and ahead of the
// sums: one after the other, each waited for, an addend cost a tile 8 us.)
template <int KIND> struct Addends {
    float4 v[4];
    __device__ __forceinline__ void load(const RaggedParams& p, int n, int k, int cols) {
        if (in_16_bits(KIND) || !p.addend || n >= p.J) return;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * j < cols && k + 4 * j < p.C)
                v[j] = *reinterpret_cast<const float4*>(p.addend + static_cast<size_t>(n) * p.C + k + 4 * j);
    }
};
// four columns k .. of row n
template <int ACT, int KIND>
__device__ __forceinline__ void store_gradient(const RaggedParams& p, int n, int k, float4 f, const float4& a) {
    if (n >= p.J || k >= p.C) return;
    const size_t at = static_cast<size_t>(n) * p.C + k;
    if (in_16_bits(KIND)) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(Act<ACT>::pack2(f.x, f.y), Act<ACT>::pack2(f.z, f.w));
    } else {
        if (p.addend) f = make_float4(f.x + a.x, f.y + a.y, f.z + a.z, f.w + a.w);
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = f;
    }
}

template <int MODE, int ACT, int KIND>
__global__ void __launch_bounds__(SPLIT_THREADS, KIND == G16LONG || KIND == G32LONG ? 2 : 1)  // (two CTAs to an SM)
split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const SplitParams sp) {
    const RaggedParams& p = sp.r;
    extern __shared__ __align__(1024) uint8_t smem[];
    SplitTail& s = *reinterpret_cast<SplitTail*>(smem + sp.tail_at);
    const WaitCtx wc{&s.abort_flag, p.err, p.wait_ns};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = sp.parts, part = parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / parts;
    const int KB = ((MODE == WGRAD ? p.rows : p.C) + BK - 1) / BK, kb0 = KB * part / parts, kb1 = KB * (part + 1) / parts;

    if (tid == 0) {
        s.abort_flag = 0;
        for (int q = 0; q < sp.stages; ++q) {
            mbar_init(&s.full[q], 1);
            mbar_init(&s.empty[q], 1);
        }
        mbar_init(&s.done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.sums[i], 1);
            mbar_init(&s.taken[i], 4);  // the epilogue's warps
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem_base, sp.tmem);
        tmem_relinquish();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
    }
    pdl_wait();
    pdl_launch_next();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    // the tile: columns j0 .. (or rows n of a gradient), rows m0 .. (columns k), n of them for the MMA
    int e = 0, j0, m0, n, rows;
    if (MODE != WGRAD && p.offsets) {
        int bad = 0;
        for (int i = tid; i < p.E; i += SPLIT_THREADS) bad |= p.offsets[i + 1] < p.offsets[i];
        if (tid == 0) bad |= p.offsets[0] < 0 || p.offsets[p.E] > p.rows;
        bad = __syncthreads_or(bad);
        if (bad && tid == 0 && blockIdx.x == 0) set_err(p.err, MOE_DEV_ERR_OFFSETS);
        const int jt = (p.J + 127) / 128;
        e = tile / jt;
        j0 = (tile - e * jt) * 128;
        m0 = p.offsets[e];
        rows = bad ? 0 : p.offsets[e + 1] - m0;
        n = (rows + 15) / 16 * 16;
    } else {
        // row tiles fastest: those of a column tile share its weights in L2
        const int i = tile % sp.mt;
        j0 = tile / sp.mt * 128;
        if (MODE == WGRAD) {
            m0 = 128 * i;
            n = rows = 128;
        } else {
            const int U = (p.rows + 15) / 16, u0 = static_cast<int>(static_cast<int64_t>(U) * i / sp.mt),
                      u1 = static_cast<int>(static_cast<int64_t>(U) * (i + 1) / sp.mt);
            m0 = 16 * u0;
            n = 16 * (u1 - u0);
            rows = min(p.rows - m0, n);
        }
    }
    const bool any = rows > 0;  // the same in all CTAs of the cluster
    const int boxes = MODE == WGRAD ? 0 : p.offsets ? n / 16 : 1;
    const uint32_t bytes = OPER + (MODE == WGRAD ? OPER : boxes * sp.box * 128), stage_bytes = sp.stage;
    // the rows of a long part of a gradient come in chunks (see gradient_chunk)
    constexpr bool CHUNKED = KIND == G16LONG || KIND == G32LONG;
    constexpr int CHUNK = gradient_chunk(!in_16_bits(KIND), ACT);
    bool ok = any;  // (a wait that gave up in another CTA of the cluster shows in the error word alone)

    if (warp == 0) {
        // ---------------- copies ----------------
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (int b = kb0; any && b < kb1; ++b) {
            if (!mbar_wait_warp(&s.empty[stage], phase ^ 1, wc)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&s.full[stage], bytes);
                uint8_t* dst = smem + stage * stage_bytes;
                if (MODE == WGRAD) {
                    tma_load_2d(dst, &tm_a, j0, b * BK, &s.full[stage]);
                    tma_load_2d(dst + 8192, &tm_a, j0 + 64, b * BK, &s.full[stage]);
                    tma_load_2d(dst + OPER, &tm_b, m0, b * BK, &s.full[stage]);
                    tma_load_2d(dst + OPER + 8192, &tm_b, m0 + 64, b * BK, &s.full[stage]);
                } else if (MODE == ROWS_FWD) {
                    load_3d(dst, &tm_a, b * BK, j0, e, &s.full[stage]);
                } else {
                    load_3d(dst, &tm_a, j0, b * BK, e, &s.full[stage]);
                    load_3d(dst + 8192, &tm_a, j0 + 64, b * BK, e, &s.full[stage]);
                }
                for (int i = 0; i < boxes; ++i)
                    tma_load_2d(dst + OPER + i * 2048, &tm_b, b * BK, m0 + 16 * i, &s.full[stage]);
            }
            __syncwarp();
            ++issued;
            if (++stage == sp.stages) {
                stage = 0;
                phase ^= 1;
            }
        }
        // let every copy land before the stages serve the sums, or the CTA exits
        for (int j = max(0, issued - sp.stages); j < issued; ++j)
            mbar_drain(&s.full[j % sp.stages], static_cast<uint32_t>((j / sp.stages) & 1), kWaitLimitNs / 8);
    } else if (warp == 1) {
        // ---------------- MMAs ----------------
        constexpr uint32_t step_a = MODE == ROWS_FWD ? 32 >> 4 : 2048 >> 4, step_b = MODE == WGRAD ? 2048 >> 4 : 32 >> 4;
        const uint32_t idesc = f16_idesc(ACT, 128, n) | (MODE == ROWS_FWD ? 0u : kMajorA) | (MODE == WGRAD ? kMajorB : 0u);
        int stage = 0;
        uint32_t phase = 0;
        for (int b = kb0; any && b < kb1; ++b) {
            uint32_t acc = tmem;
            bool more = b > kb0;  // adds to what the accumulator holds
            if constexpr (CHUNKED) {  // the two accumulators in turn
                const int ch = (b - kb0) / CHUNK, in = (b - kb0) - ch * CHUNK;
                if (in == 0 && ch > 0) {
                    if (elect_one()) tc_commit(&s.sums[(ch - 1) & 1]);
                    __syncwarp();
                    if (ch > 1) {
                        if (!mbar_wait_warp(&s.taken[ch & 1], ((ch >> 1) - 1) & 1, wc)) break;
                        tc_fence_after();
                    }
                }
                acc += (ch & 1) * 128;
                more = in > 0;
            }
            if (!mbar_wait_warp(&s.full[stage], phase, wc)) break;
            tc_fence_after();
            const uint32_t at = smem_u32(smem + stage * stage_bytes);
            const uint64_t ad = MODE == ROWS_FWD ? sw128_desc(at) : mn_desc(at);
            const uint64_t bd = MODE == WGRAD ? mn_desc(at + OPER) : sw128_desc(at + OPER);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    tc_mma(acc, ad + k * step_a, bd + k * step_b, idesc, more || k > 0);
                tc_commit(&s.empty[stage]);
            }
            __syncwarp();
            if (++stage == sp.stages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (elect_one()) tc_commit(&s.done);
        __syncwarp();
        mbar_drain(&s.done, 0, kWaitLimitNs / 8);
    } else {
        if constexpr (KIND == FULL) prefetch_residual(p, lane, m0, rows, j0 + 32 * (warp & 3));
        if constexpr (CHUNKED) {
            // the chunks' sums, added up in registers and laid into the first accumulator
            const int chunks = (kb1 - kb0 + CHUNK - 1) / CHUNK;
            const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            uint32_t v[8][16];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[i][j] = 0u;
            for (int ch = 0; ch < chunks; ++ch) {
                const bool last = ch + 1 == chunks;
                ok = mbar_wait_warp(last ? &s.done : &s.sums[ch & 1], last ? 0 : ch >> 1 & 1, wc);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t u[16];
                    tmem_ld16(lanes + (ch & 1) * 128 + 16 * i, u);
                    tmem_ld16_wait(u);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[i][j] = __float_as_uint(__uint_as_float(v[i][j]) + __uint_as_float(u[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !last) mbar_arrive(&s.taken[ch & 1]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) tmem_st16(lanes + 16 * i, v[i]);
            tmem_st_wait();
        } else {
            ok = mbar_wait_warp(&s.done, 0, wc) && any;
            tc_fence_after();
        }
    }
    __syncwarp();
    const bool epi = warp >= 2;
    const int q = warp & 3, me = 32 * q + lane;
    const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const float bias = KIND == FULL && epi ? bias_of<ACT>(p, j0 + me) : 0.0f;
    // the epilogue's areas lie where the stages were: the sums of all parts, then staging
    const int sum_bytes = parts > 1 ? parts * ((n / 4 + parts - 1) / parts) * 2048 : 0;  // (slices may differ by 4 rows)
    float* stg = reinterpret_cast<float*>(smem + sum_bytes + (warp - 2) * (STG_ROWS * SG * 4));
    if (parts == 1) {
        if (epi && ok)
#pragma unroll 1
            for (int c = 0; c < rows; c += 16) {
                uint32_t u[16];
                float v[16];
                Residual res;
                Addends<KIND> add;
                if (KIND == FULL) res.load(p, lane, m0 + c, rows - c, j0 + 32 * q);
                if (MODE == WGRAD) add.load(p, j0 + me, m0 + c, 16);
                tmem_ld16(ta + c, u);
                tmem_ld16_wait(u);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(u[j]) + bias;
                if constexpr (MODE == WGRAD) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        store_gradient<ACT, KIND>(p, j0 + me, m0 + c + j, make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]),
                                                  add.v[j / 4]);
                } else {
                    store_rows<ACT, KIND>(p, v, res, stg, lane, m0 + c, rows - c, j0 + 32 * q);
                }
            }
    } else if (any) {
        cluster_sync_all();  // every CTA's MMAs are complete: the stages are free
        // part d adds rows 4 f(d) to 4 f(d + 1), f(d) = n / 4 d / parts: four rows of a column are a 16-byte store.
        // There, [source part][four rows][128 columns][4]
        float4* sums = reinterpret_cast<float4*>(smem);
        const int quads = n / 4;
        if (epi) {
            int dst = 0, f0 = 0, f1 = quads / parts;
            while (f1 == f0) f1 = quads * (++dst + 1) / parts;
            const uint32_t mine = smem_u32(sums + me);
            uint32_t to = mapa_shared(mine + part * (f1 - f0) * 2048, dst);
#pragma unroll 1
            for (int c = 0; c < n; c += 16) {
                uint32_t u[16];
                tmem_ld16(ta + c, u);
                tmem_ld16_wait(u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int f = c / 4 + j;
                    if (f == f1) {
                        f0 = f1;
                        while (f1 == f0) f1 = quads * (++dst + 1) / parts;
                        to = mapa_shared(mine + part * (f1 - f0) * 2048, dst);
                    }
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (f - f0) * 2048),
                                 "r"(u[4 * j]), "r"(u[4 * j + 1]), "r"(u[4 * j + 2]), "r"(u[4 * j + 3])
                                 : "memory");
                }
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (epi && ok) {
            const int q0 = quads * part / parts, per = quads * (part + 1) / parts - q0;
            const int have = min(4 * per, rows - 4 * q0);
#pragma unroll 1
            for (int c = 0; c < have; c += 16) {
                float v[16];
                Residual res;
                Addends<KIND> add;
                if (KIND == FULL) res.load(p, lane, m0 + 4 * q0 + c, have - c, j0 + 32 * q);
                if (MODE == WGRAD) add.load(p, j0 + me, m0 + 4 * q0 + c, have - c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (c + 4 * j < have) {
                        const float4* src = sums + (c / 4 + j) * 128 + me;
                        f = src[0];
                        for (int r = 1; r < parts; ++r) {
                            const float4 x = src[r * per * 128];
                            f.x += x.x;
                            f.y += x.y;
                            f.z += x.z;
                            f.w += x.w;
                        }
                    }
                    if constexpr (MODE == WGRAD) {
                        if (c + 4 * j < have) store_gradient<ACT, KIND>(p, j0 + me, m0 + 4 * q0 + c + 4 * j, f, add.v[j]);
                    }
                    v[4 * j] = f.x + bias;
                    v[4 * j + 1] = f.y + bias;
                    v[4 * j + 2] = f.z + bias;
                    v[4 * j + 3] = f.w + bias;
                }
                if constexpr (MODE != WGRAD)
                    store_rows<ACT, KIND>(p, v, res, stg, lane, m0 + 4 * q0 + c, have - c, j0 + 32 * q);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, sp.tmem);
}

// Three stages hold the sums (2048 bytes for four rows of each part, the largest slice counting for all) and the
// staging areas: of 128 rows as of 16.
constexpr int split_sums(int n) { return SPLIT_PARTS * ((n / 4 + SPLIT_PARTS - 1) / SPLIT_PARTS) * 2048; }
static_assert(3 * (OPER + SPLIT_ROWS * 128) >= split_sums(SPLIT_ROWS) + 4 * STG_ROWS * SG * 4 &&
                  3 * (OPER + 16 * 128) >= split_sums(16) + 4 * STG_ROWS * SG * 4 &&
                  3 * (OPER + 48 * 128) >= split_sums(48) + 4 * STG_ROWS * SG * 4,
              "the epilogue's areas fit in the stages");

// tiles: clusters of the grid; mt as in SplitParams
template <int MODE, int ACT, int KIND> int launch_split_kind(const RaggedArgs& g, int64_t tiles, int mt, int parts) {
    auto kernel = split_kernel<MODE, ACT, KIND>;
    // of shared memory: two CTAs to an SM, or all where there are fewer CTAs than SMs (clusters of 8 with an SM
    // each do not fill the GPU: 128 CTAs of 2048 columns take 11.8 us so, two to an SM 7.5)
    constexpr int all = 229376, half = 114688;
    const int most = parts < 8 && tiles * parts * 10 <= sm_count() * 9 ? all : half;
    static PerDevice configured;
    int rc = raise_smem_limit(configured, reinterpret_cast<const void*>(kernel), all);
    if (rc != MOE_OK) return rc;
    SplitParams sp;
    sp.r = g.p;
    sp.parts = parts;
    sp.mt = mt;
    const int rows = MODE == WGRAD ? SPLIT_ROWS : ((g.p.rows + 15) / 16 + mt - 1) / mt * 16;  // of the tallest tile
    sp.box = MODE == WGRAD ? 64 : g.p.offsets ? 16 : rows;
    sp.tmem = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    if (KIND == G16LONG || KIND == G32LONG) sp.tmem = 256;  // two accumulators
    const int rest = static_cast<int>(sizeof(SplitTail));
    sp.stage = OPER + rows * 128;
    sp.stages = (most - rest) / sp.stage;  // 3 at least
    if (sp.stages > SPLIT_MAX_STAGES) sp.stages = SPLIT_MAX_STAGES;
    sp.tail_at = sp.stages * sp.stage;
    Maps m;
    if (MODE == WGRAD) {
        rc = make_tmap_2d(&m.a, g.a, g.p.rows, g.N, 64, g.act);
        if (rc == MOE_OK) rc = make_tmap_2d(&m.b, g.w, g.p.rows, g.K, 64, g.act);
    } else {
        rc = make_tmap_3d(&m.a, const_cast<void*>(g.w), g.act, g.K, g.N, g.p.E, 64, MODE == ROWS_FWD ? 128 : 64);
        if (rc == MOE_OK) rc = make_tmap_2d(&m.b, g.a, g.p.rows, g.p.C, sp.box, g.act);
    }
    if (rc != MOE_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * parts));
    cfg.blockDim = dim3(SPLIT_THREADS);
    cfg.dynamicSmemBytes = sp.tail_at + rest;
    cfg.stream = g.st;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, sp);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", g.who, cudaGetErrorString(e));
    count_launch();
    return check_launch(g.who);
}

// row tiles of one group, or every group with a tile
template <int MODE, int ACT> int launch_split(const RaggedArgs& g, int mt, int parts) {
    const int64_t tiles = static_cast<int64_t>((g.p.J + 127) / 128) * (g.p.offsets ? g.p.E : mt);
    if (MODE == ROWS_FWD && (g.p.bias || g.p.residual || g.p.pre || g.p.fn != MOE_FN_NONE))
        return launch_split_kind<ROWS_FWD, ACT, FULL>(g, tiles, mt, parts);
    return launch_split_kind<MODE, ACT, PLAIN>(g, tiles, mt, parts);
}

// A product of rows in the form that was chosen for it.
template <int ACT> int launch_rows_act(const RaggedArgs& g, const RowsForm& f) {
    if (f.parts)
        return g.transposed ? launch_split<ROWS_BACK, ACT>(g, f.tiles, f.parts)
                            : launch_split<ROWS_FWD, ACT>(g, f.tiles, f.parts);
    return g.transposed ? launch_rows_form<ROWS_BACK, ACT>(g, f.maxu) : launch_rows_form<ROWS_FWD, ACT>(g, f.maxu);
}

}  // namespace
}  // namespace ragged
}  // namespace moe
