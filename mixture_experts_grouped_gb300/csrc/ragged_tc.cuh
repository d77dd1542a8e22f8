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
//   A tile is 256 rows n by up to 256 columns k. Both operands are MN-major, the contraction
//   runs over the group's rows: whole units of 16, four to a block. The rows that are left,
//   1 to 15, are a unit of their own: its other rows belong to the next group or to nobody
//   (they may hold infinities), so a warp of each CTA has the unit copied into a buffer
//   apart, sets those rows to zeros in both operands, and then lets the MMA have it. The
//   buffers are two, filled up to two tiles ahead: in the ring of blocks, where a unit is
//   copied only six blocks before its MMA, the way from its arrival over the clearing to
//   the other CTA's MMA warp was not hidden and cost 1.2 us a tile (8 groups of 1024 rows,
//   4096 x 14336: 668 us, 559 with rows that 16 divides).
//
// Roles: warps 0 and 2 copy the two operands (TMA, 128-byte swizzle), warp 1 of the even
// CTA (the leader) issues the MMAs, warp 3 makes the tails, warps 4 to 11 are the epilogue
// (GADD: the latter four copy for the former).
// Two accumulators of 256 TMEM columns let the epilogue of a tile run beside the next
// one's MMAs. The issuing warps run their loops whole and elect a lane for the MMAs and
// copies: by a lane that a branch on the lane number singled out, each took longer (4096 x
// 14336 x 4096: 271 us, 245 elected). Every wait is bounded.
//
// Measured: 8192 rows of 8 groups, 28672 x 4096 1014 to 1066 us, 1.8 to 1.9 PFLOP/s (1166 to 1224
// under the power cap of long runs); its transposed form the same; 64 rows of 50 touched
// groups, 1536 x 2048 55 us, 5.7 TB/s. Gradients: 8192 rows of 8 groups, 4096 x 14336 bf16 545 us,
// 1.76 PFLOP/s; 12288 rows of 64 groups, 2048 x 1408 f32 with addends 234 us, 6.6 TB/s; 32768 rows
// of 128 groups, 1536 x 2048 bf16 184 us, 5.6 TB/s.
#pragma once

#include <numeric>

#include "ragged.cuh"

namespace moe {
namespace ragged {
// (in a namespace of its own file: every .cu that includes this has its own kernels)
namespace {

enum { ROWS_FWD = 0, ROWS_BACK = 1, WGRAD = 2 };
// kinds of gradient: 16-bit, f32, f32 with addends that come by TMA (GADD) or by loads (G32ADD; ragged_wgrad.cu has the
// choice), and those whose chunks' loop would cost the others time or registers: 16-bit of more rows than a chunk, and
// (split form alone) f32; of the rows form: the product alone, or with bias, activation function, residual and z (their
// code, jumped over, still cost a plain product's epilogue half its time in instruction fetches)
enum { G16 = 0, G32 = 1, GADD = 2, G16LONG = 4, G32LONG = 5, G32ADD = 6, PLAIN = 0, FULL = 3 };
constexpr bool in_16_bits(int kind) { return kind == G16 || kind == G16LONG; }
constexpr bool in_registers(int kind) { return kind == G32 || kind == G32ADD; }  // (see RowSums)

constexpr int BK = 64;
constexpr int OPER = 128 * BK * 2;  // bytes of a CTA's share of an operand per stage
constexpr int STAGE = 2 * OPER;
constexpr int MAX_STAGES = 10;
constexpr int STG = 32 * 64;  // rows form: a warp's staging area
constexpr int UNIT = 64 * 16 * 2;             // gradient form: 64 columns of a unit of 16 rows
constexpr int TBUF = 4 * UNIT, TBUFS = 2;     // a tail of both operands
constexpr int SLOT = 32 * 128;                // gradient form: 32 rows x 128 bytes of dw

struct Tail {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t tloc[TBUFS], tready[TBUFS], tfree[TBUFS];  // tails: copied (this CTA's), cleared (both CTAs'), used
    uint64_t tfull[2], tempty[2], mma_done;
    uint64_t slot[4][4], sdone[4][4];  // a warp's slots: addend there, sums there
    uint32_t tmem_base;
    int abort_flag, n_tiles, jt;
    int off[MOE_MAX_EXPERTS + 1];
    int tstart[MOE_MAX_EXPERTS + 1];
};

// Epilogue warps, and shared memory: the ring of stages, tails, staging areas. Eight
// warps finish a tile, two to a quarter of the TMEM lanes, which take its steps in turn. A
// gradient with an addend is bound by their bytes: four warps with four slots each, so that
// three steps' addends are on their way, four others that load and store for them, and
// four stages. Other gradients have a slot a warp and five stages (8192 rows, 8 groups, 4096 x
// 14336: 557 us, 631 with four). The rows form has six stages of full height, more of lower
// ones: a group's few rows leave a tile to its weights' latency, and an SM streams them as
// fast as it has copies in flight.
template <int MODE, int KIND> struct Shape {
    static constexpr int HALVES = KIND == GADD ? 1 : 2;  // warps to a quarter
    static constexpr int WARPS = 4 * HALVES;
    static constexpr int THREADS = 384;
    // kinds that keep a tile's sums in registers: those of the first four warps' threads, and of the epilogue's; together
    // no more than the launch's
    static constexpr int REGS_ROLES = 72, REGS_SUMS = 216, REGS_LAUNCH = 168;
    static_assert(128 * REGS_ROLES + 256 * REGS_SUMS <= THREADS * REGS_LAUNCH, "more registers than the launch has");
    static constexpr int SLOTS = KIND == GADD ? 4 : 1;
    static constexpr int STAGES = MODE != WGRAD ? 6 : KIND == GADD ? 4 : 5;  // of full height
    static constexpr int STG_WARP = MODE == WGRAD ? SLOTS * SLOT : STG;
    static constexpr int TBUF_AT = STAGES * STAGE;
    static constexpr int STG_AT = TBUF_AT + (MODE == WGRAD ? TBUFS * TBUF : 0);
    static constexpr int TAIL_AT = STG_AT + WARPS * STG_WARP;
    static constexpr int SMEM = TAIL_AT + (static_cast<int>(sizeof(Tail)) + 127) / 128 * 128;
    static_assert(SMEM <= 232448, "shared memory over the limit");
};

// stages that the ring's bytes hold
template <int MODE, int KIND> __device__ __forceinline__ uint32_t n_stages(uint32_t stage_bytes) {
    return min(static_cast<uint32_t>(MAX_STAGES), Shape<MODE, KIND>::STAGES * STAGE / stage_bytes);
}

// ---- operands -------------------------------------------------------------------------
// MN-major operand with the 128-byte swizzle, as a TMA box of 64 elements (128 bytes) x 64
// contraction indices lays it down: 8 contraction indices are 1024 bytes (the stride
// offset), the next 64 elements are 8192 bytes on (the leading offset).
// (A unit's box has 16 indices, so its next 64 elements are 2048 bytes on.)
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t lead = 8192u) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
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
// all but this thread's last group have read their shared memory
__device__ __forceinline__ void store_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Arrival on a barrier of the other CTA, ordered after this thread's work on its own CTA's
// shared and tensor memory, which is all that these signals are about (the tensor core
// reads each CTA's own). A release at cluster scope also waits for what the thread stored to
// global memory, and held up the next tile's MMAs by about 1 us.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- tiles ------------------------------------------------------------------------------
struct Tile {
    int e;
    int j0;        // rows form: first output column; gradient form: first n
    int m0, rows;  // rows form: first row and rows of the tile; gradient form: the group's
    int n;         // the MMA's N
    int k0;        // gradient form: first k
};

// x / d of x >= 0, d > 0, by an approximate quotient: off by one below 2^24, by a few above
__device__ __forceinline__ int quotient(int x, int d) {
    int q = __float2int_rz(__fdividef(static_cast<float>(x), static_cast<float>(d)));
    int r = x - q * d;
    while (r < 0) --q, r += d;
    while (r >= d) ++q, r -= d;
    return q;
}

// Rows form: a group's rows are cut into tiles of nearly equal height, in units of 16 rows
// and at most maxu of them. Every CTA builds the list from the offsets: the tiles of group
// e begin at tstart[e], its row tiles fastest, then output columns. Returns whether the
// offsets are bad (no tile then).
template <int MODE>
__device__ __forceinline__ int build_tiles(Tail& s, const RaggedParams& p) {
    const int tid = threadIdx.x, lane = tid & 31, E = p.E;
    for (int i = tid; i <= E; i += blockDim.x) s.off[i] = p.offsets ? p.offsets[i] : (i ? p.rows : 0);
    const int jt = (p.J + 255) / 256;
    if (tid == 0) {
        s.abort_flag = 0;
        s.jt = jt;
    }
    __syncthreads();
    int bad = 0;
    for (int i = tid; i < E; i += blockDim.x) bad |= s.off[i + 1] < s.off[i];
    if (tid == 0) bad |= s.off[0] < 0 || s.off[E] > p.rows;
    bad = __syncthreads_or(bad);
    if (MODE == WGRAD) {
        if (tid == 0) s.n_tiles = bad ? 0 : E * static_cast<int>(p.per.d);
        return bad;
    }
    if (tid < 32) {
        auto tiles = [&](int e) {
            return e < E && !bad ? p.units.div((s.off[e + 1] - s.off[e] + 15) / 16 + p.maxu - 1) * jt : 0;
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
        t.e = p.per.div(tile);
        const int in = tile - t.e * static_cast<int>(p.per.d), jn = p.kt.div(in), kn = in - jn * static_cast<int>(p.kt.d);
        t.j0 = jn * 256;
        t.k0 = (kn * p.kleast + min(kn, p.kmore)) * p.kunit;
        t.m0 = s.off[t.e];
        t.rows = s.off[t.e + 1] - t.m0;
        t.n = (p.kleast + (kn < p.kmore)) * p.kunit;
        return t;
    }
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.tstart[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    // (of groups that begin at the same tile all but the last are empty)
    t.e = lo;
    const int v = s.off[lo + 1] - s.off[lo], U = (v + 15) / 16, mt = p.units.div(U + p.maxu - 1);
    const int local = tile - s.tstart[lo], jn = quotient(local, mt), i = local - jn * mt;
    const int least = quotient(U, mt), u0 = i * least + min(i, U - mt * least);  // the first tiles take a unit more
    const int units = least + (i < U - mt * least);
    t.m0 = s.off[lo] + 16 * u0;
    t.rows = min(v - 16 * u0, 16 * units);
    t.n = 16 * units;
    t.j0 = jn * 256;
    t.k0 = 0;
    return t;
}

// A pair's tiles: one of every wave, `turn` places on in each, so that the narrow tiles at the edges, which come at
// regular distances, are not all dealt to the same pairs (15421 rows of 133 groups, 3784 x 288 f32 with addends, tiles of
// 160 and 128 columns side by side: 196 us, 230 without).
struct Walk {
    int tile, pos, step, turn;
    __device__ __forceinline__ explicit Walk(const RaggedParams& p)
        : tile(blockIdx.x >> 1), pos(tile), step(gridDim.x >> 1), turn(p.turn) {}
    __device__ __forceinline__ void next() {
        tile += step + turn;
        pos += turn;
        if (pos >= step) {
            pos -= step;
            tile -= step;
        }
    }
};

// ---- epilogues --------------------------------------------------------------------------

// Rows form: how a warp's rows x 32 columns lie in memory, as 16-byte pieces of 8 columns: lane l has pieces of
// rows l / 4, 8 + l / 4 and so on.
struct Piece {
    int r, col;
    __device__ __forceinline__ Piece(int i, int lane, int col0) : r(8 * i + (lane >> 2)), col(col0 + 8 * (lane & 3)) {}
    __device__ __forceinline__ bool in(const RaggedParams& p, int rows) const { return r < rows && col < p.J; }
    __device__ __forceinline__ size_t at(const RaggedParams& p, int m) const {
        return static_cast<size_t>(m + r) * p.J + col;
    }
};
// brings the residual of rows m .. m + rows - 1 into L2, ahead of its use
__device__ __forceinline__ void prefetch_residual(const RaggedParams& p, int lane, int m, int rows, int col0) {
    if (!p.residual) return;
    for (int r = lane >> 1; r < rows; r += 16) {
        const int col = col0 + 16 * (lane & 1);
        if (col < p.J)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.residual + static_cast<size_t>(m + r) * p.J + col));
    }
}

// 16 columns of the accumulator
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int ACT>
__device__ __forceinline__ float bias_of(const RaggedParams& p, int col) {
    if (!p.bias || col >= p.J) return 0.0f;
    return Act<ACT>::to_f(reinterpret_cast<const typename Act<ACT>::T*>(p.bias)[col]);
}

// 8 U columns of 16 lanes, as the fragments of 8 x 8 matrices: register 4 u + 2 k + i is lane 8 k + T / 4, column 8 u +
// 2 (T % 4) + i, T the thread
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
template <int N> __device__ __forceinline__ void tmem_ld_frag_wait(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A warp's staging area: rows of 32 columns in 16 bits; the four 16-byte pieces of a row are swizzled by row pairs, so
// that neither eight rows of a piece nor the pieces of two rows meet in a bank.
__device__ __forceinline__ uint32_t piece_at(uint32_t stg, int r, int piece) {
    return stg + r * 64 + ((piece ^ (r >> 1 & 3)) << 4);
}
// fragments (lane j, rows m) to the area, transposed: row m, columns j
template <int U> __device__ __forceinline__ void stage_frags(uint32_t stg, int lane, const uint32_t (&f)[U][4]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         piece_at(stg, 8 * u + (lane & 7), lane >> 3)),
                     "r"(f[u][0]), "r"(f[u][1]), "r"(f[u][2]), "r"(f[u][3])
                     : "memory");
}
// the area's rows to memory: 16-byte pieces, eight rows at a time
template <int U>
__device__ __forceinline__ void copy_rows(const RaggedParams& p, uint16_t* out, uint32_t stg, int lane, int m, int rows,
                                          int col0) {
    __syncwarp();
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "r"(piece_at(stg, 8 * i + (lane >> 2), lane & 3))
                     : "memory");
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const Piece c(i, lane, col0);
        if (c.in(p, rows)) *reinterpret_cast<uint4*>(out + c.at(p, m)) = v[i];
    }
    __syncwarp();
}

// Rows form: a warp's 32 columns (TMEM lanes) of a tile, a step of rows at a time, every other step. The sums are read as
// fragments, finished in f32, rounded, and turned in the staging area. (By one lane a column, with f32 values staged, a
// plain tile of 256 rows took 2.5 us, now 1.9: 8192 x 8192 x 64 43 us and 33.) A step is 32 rows of a plain product; 16 with
// bias, function or residual, whose code is twice as long.
template <int ACT, int KIND>
__device__ __forceinline__ void rows_epilogue(const RaggedParams& p, uint32_t ta, uint32_t stg, const Tile& t, int col0,
                                              int half, int lane) {
    constexpr int U = KIND == FULL ? 2 : 4, STEP = 8 * U;
    float b[4];  // of lanes 8 j + T / 4
    if (KIND == FULL)
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = bias_of<ACT>(p, col0 + 8 * j + (lane >> 2));
    uint32_t nx[2][4 * U];
    uint4 res[U];
    auto load = [&](int c) {
        tmem_ld_frag(ta + c, nx[0]);
        tmem_ld_frag(ta + (16u << 16) + c, nx[1]);
        if (KIND != FULL || !p.residual) return;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const Piece q(i, lane, col0);
            if (q.in(p, t.rows - c)) res[i] = *reinterpret_cast<const uint4*>(p.residual + q.at(p, t.m0 + c));
        }
    };
    if (STEP * half < t.rows) load(STEP * half);
#pragma unroll 1
    for (int c = STEP * half; c < t.rows; c += 2 * STEP) {
        float v[U][8];  // [eight rows][two rows of a lane's four columns]
        uint32_t f[U][4], r[U][4];
        tmem_ld_frag_wait(nx[0]);
        tmem_ld_frag_wait(nx[1]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[u][j] = __uint_as_float(nx[j >> 2][4 * u + (j & 3)]);
                if (KIND == FULL) v[u][j] += b[j >> 1];
            }
        if (KIND == FULL && p.residual) {  // to the area, and back as fragments
#pragma unroll
            for (int i = 0; i < U; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 piece_at(stg, 8 * i + (lane >> 2), lane & 3)),
                             "r"(res[i].x), "r"(res[i].y), "r"(res[i].z), "r"(res[i].w)
                             : "memory");
            __syncwarp();
#pragma unroll
            for (int u = 0; u < U; ++u)
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r[u][0]), "=r"(r[u][1]), "=r"(r[u][2]), "=r"(r[u][3])
                             : "r"(piece_at(stg, 8 * u + (lane & 7), lane >> 3))
                             : "memory");
            __syncwarp();
        }
        if (c + 2 * STEP < t.rows) load(c + 2 * STEP);  // in flight while this one is finished
        auto round_all = [&] {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[u][j] = Act<ACT>::pack2(v[u][2 * j], v[u][2 * j + 1]);
        };
        if (KIND == FULL && p.pre) {
            round_all();
            stage_frags(stg, lane, f);
            copy_rows<U>(p, p.pre, stg, lane, t.m0 + c, t.rows - c, col0);
        }
        if (KIND == FULL) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                fn_values(p.fn, v[u]);
                if (!p.residual) continue;
                float g[8];
                unpack8<ACT>(make_uint4(r[u][0], r[u][1], r[u][2], r[u][3]), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] += g[j];
            }
        }
        round_all();
        stage_frags(stg, lane, f);
        copy_rows<U>(p, static_cast<uint16_t*>(p.out), stg, lane, t.m0 + c, t.rows - c, col0);
    }
}

// A tensor core's f32 sums are cut, not rounded, at each step of 16 products: of n products
// of one sign, a sum comes out up to n 2^-27 short (measured, as a part of it: 4096 rows
// 2.6e-5, 30000 1.9e-4), and of n products of random signs n 1.2e-9. A gradient therefore
// takes its rows in chunks (gradient_chunk) and adds the chunks in f32. G32 and G32ADD: the
// chunks take the accumulators in turn, and the epilogue adds them up in registers, 128 a
// lane, beside the next chunk's MMAs (16384 rows of 8 groups, 4096 x 3584 f32: 282 us, 275 with
// 4096 rows in one accumulator; 1333 rows, 2816 x 2048: 20.0 and 19.0). GADD, whose groups are
// short, and G16LONG: the first chunk stays in its accumulator, the others come into the second
// one and are added to it, the last one on its way out.

// adds the accumulator at tb to the one at ta: the columns that this warp will store, COLS of
// every HALVES * COLS
template <int COLS, int HALVES> __device__ __forceinline__ void fold(uint32_t ta, uint32_t tb, int half) {
#pragma unroll 1
    for (int c = half * COLS; c < 256; c += HALVES * COLS) {
#pragma unroll 1
        for (int i = c; i < c + COLS; i += 32) {
            uint32_t u[32], v[32];
            tmem_ld32(ta + i, u);
            tmem_ld32(tb + i, v);
            tmem_ld_wait_regs(u);
            tmem_ld_wait_regs(v);
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) + __uint_as_float(v[j]));
            tmem_st32(ta + i, u);
        }
    }
    tmem_st_wait();
}

// Gradient form: lane = row n of dw, columns k. A step is 128 bytes of each row (32 f32 or
// 64 16-bit values): they are laid into one of the warp's slots, 16-byte pieces swizzled by
// row, and leave by a TMA store, which leaves out what lies past the weight's edges. An
// addend comes into the slot by a TMA load three steps before and is added in place.
template <int KIND> struct Slots {
    static constexpr int COLS = in_16_bits(KIND) ? 64 : 32;
    static constexpr int N = Shape<WGRAD, KIND>::SLOTS;
};

__device__ __forceinline__ int tile_cols(const RaggedParams& p, const Tile& t) { return min(t.n, p.C - t.k0); }

// With an addend: the copies of one epilogue warp's slots. They are a warp of their own
// because finding, waiting for and issuing them took as long as the sums (a step 0.9 us,
// all by one warp).
__device__ __forceinline__ void copy_slots(Tail& s, const RaggedParams& p, const CUtensorMap* tm_out,
                                           const CUtensorMap* tm_add, uint8_t* area, int w, int n_off, int n_tiles,
                                           int lane, const WaitCtx& wc) {
    constexpr int N = Slots<GADD>::N, COLS = Slots<GADD>::COLS;
    Walk at(p), lat(p);
    if (at.tile >= n_tiles) return;
    int lc = 0;  // the next load's column
    uint32_t loaded = 0, stored = 0;
    Tile lt = get_tile<WGRAD>(s, p, lat.tile), t = lt;
    auto load = [&] {
        if (lat.tile >= n_tiles) return;
        const uint32_t i = loaded % N;
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.slot[w][i], SLOT);
            tma_load_3d(area + i * SLOT, tm_add, lt.k0 + lc, lt.j0 + n_off, lt.e, &s.slot[w][i]);
        }
        __syncwarp();
        ++loaded;
        lc += COLS;
        if (lc >= tile_cols(p, lt)) {
            lc = 0;
            lat.next();
            if (lat.tile < n_tiles) lt = get_tile<WGRAD>(s, p, lat.tile);
        }
    };
    for (int i = 0; i < N - 1; ++i) load();
    bool ok = true;
    for (; at.tile < n_tiles && ok; at.next()) {
        t = get_tile<WGRAD>(s, p, at.tile);
        const int cols = tile_cols(p, t);
        for (int c = 0; c < cols; c += COLS) {
            const uint32_t i = stored % N;
            if (!mbar_wait_warp(&s.sdone[w][i], (stored / N) & 1u, wc)) {
                ok = false;
                break;
            }
            ++stored;
            if (lane == 0) {
                if (t.j0 + n_off < p.J) store_3d(tm_out, area + i * SLOT, t.k0 + c, t.j0 + n_off, t.e);
                store_commit();       // one group a step, empty or not
                store_wait_read1();   // the step before has been read: its slot takes the next load
            }
            __syncwarp();
            load();
        }
    }
    if (lane == 0) {
        // (loads that nobody waited for are left only after a wait that gave up)
        for (uint32_t i = loaded > N ? loaded - N : 0; i < loaded; ++i)
            mbar_drain(&s.slot[w][i % N], (i / N) & 1u, kWaitLimitNs / 8);
        store_wait();
    }
    __syncwarp();
}

template <int ACT>
__device__ __forceinline__ uint4 pack_piece(const float* v) {
    return make_uint4(Act<ACT>::pack2(v[0], v[1]), Act<ACT>::pack2(v[2], v[3]), Act<ACT>::pack2(v[4], v[5]),
                      Act<ACT>::pack2(v[6], v[7]));
}

// 32 columns of the sums: none of an empty group, of one accumulator or of two
__device__ __forceinline__ void load_sums(uint32_t ta, uint32_t tb, int accs, float (&v)[32]) {
    if (accs == 0) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        return;
    }
    uint32_t u[32];
    tmem_ld32(ta, u);
    tmem_ld_wait_regs(u);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
    if (accs > 1) {
        tmem_ld32(tb, u);
        tmem_ld_wait_regs(u);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(u[j]);
    }
}

// A tile's sums, in the accumulator at ta and, with accs 2, the one at tb. `used` counts the
// warp's steps. Returns false if a wait gave up.
template <int ACT, int KIND>
__device__ __forceinline__ bool wgrad_epilogue(Tail& s, const RaggedParams& p, const CUtensorMap* tm_out, uint8_t* area,
                                               uint32_t& used, uint32_t ta, uint32_t tb, int accs, const Tile& t, int w,
                                               int n_off, int half, int lane, const WaitCtx& wc) {
    constexpr int COLS = Slots<KIND>::COLS, N = Slots<KIND>::N, HALVES = Shape<WGRAD, KIND>::HALVES;
    const int cols = tile_cols(p, t);
#pragma unroll 1
    for (int c = half * COLS; c < cols; c += HALVES * COLS) {
        float v[32];
        load_sums(ta + c, tb + c, accs, v);
        const uint32_t i = used % N;
        uint8_t* at = area + i * SLOT + lane * 128;
        if (KIND == GADD) {
            if (!mbar_wait_warp(&s.slot[w][i], (used / N) & 1u, wc)) return false;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 f = *reinterpret_cast<const float4*>(at + 16 * (q ^ (lane & 7)));
                v[4 * q] += f.x;
                v[4 * q + 1] += f.y;
                v[4 * q + 2] += f.z;
                v[4 * q + 3] += f.w;
            }
        } else {
            if (lane == 0) store_wait_read();  // the slot's last store
            __syncwarp();
        }
        ++used;
        if (in_16_bits(KIND)) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(at + 16 * (q ^ (lane & 7))) = pack_piece<ACT>(v + 8 * q);
            load_sums(ta + c + 32, tb + c + 32, accs, v);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(at + 16 * ((4 + q) ^ (lane & 7))) = pack_piece<ACT>(v + 8 * q);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4*>(at + 16 * (q ^ (lane & 7))) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (KIND == GADD) {
                mbar_arrive(&s.sdone[w][i]);
            } else if (t.j0 + n_off < p.J) {
                store_3d(tm_out, area + i * SLOT, t.k0 + c, t.j0 + n_off, t.e);
                store_commit();
            }
        }
    }
    return true;
}

// ---- G32, G32ADD: sums in registers ----------------------------------------------------------------
// Lane = row n of dw; a warp has every other 32 columns of a tile.
struct RowSums {
    uint32_t v[4][32];
    // adds 32 columns of an accumulator
    __device__ __forceinline__ void add(int i, uint32_t ta) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t u[16];
            tmem_ld16(ta + 16 * h, u);
            tmem_ld16_wait(u);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[i][16 * h + j] = __float_as_uint(__uint_as_float(v[i][16 * h + j]) + __uint_as_float(u[j]));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[i][j] = 0u;
    }
};
// brings the lane's addends into L2, ahead of their use
__device__ __forceinline__ void prefetch_addend(const RaggedParams& p, const Tile& t, int row, int first, int cols) {
    if (t.j0 + row >= p.J) return;
    const float* at = p.addend + (static_cast<size_t>(t.e) * p.J + t.j0 + row) * p.C + t.k0;
    for (int c = first; c < cols; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c));
}
// A warp's sums, and its addends, through its slot to dw (which may hold the addends). The
// addends are read 128 bytes of a row to eight lanes, a step ahead, and meet the sums in the
// slot: read by the lane that adds them, they took the L1 1.1 us a step of the CTA's warps
// (16384 rows of 8 groups, 4096 x 3584: 395 us, so 346).
struct Addend {
    float4 f[8];  // of rows 4 q + lane / 8
    __device__ __forceinline__ void load(const float* at, int C, int rows, int cols, int lane) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r = 4 * q + (lane >> 3), c = 4 * (lane & 7);
            f[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows && c < cols) f[q] = *reinterpret_cast<const float4*>(at + static_cast<size_t>(r) * C + c);
        }
    }
};
template <int KIND>
__device__ __forceinline__ void store_sums(const RaggedParams& p, const CUtensorMap* tm_out, uint8_t* slot, RowSums& s,
                                           uint32_t ta, const Tile& t, int n_off, int half, int cols, int lane) {
    const int n = t.j0 + n_off;
    const float* from = p.addend + (static_cast<size_t>(t.e) * p.J + n) * p.C + t.k0;
    // (G32ADD always has them. Where the compiler knows, it issues the next step's loads too
    // late: 8192 rows of 8 groups, 4096 x 3584, 231 us and 222)
    const bool add = KIND == G32ADD && p.addend;
    Addend a;
    if (add) a.load(from + 32 * half, p.C, p.J - n, cols - 32 * half, lane);
    uint8_t* at = slot + lane * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = 32 * half + 64 * i;
        if (c >= cols) break;
        if (KIND == G32 && t.rows > 0) s.add(i, ta + 64 * i);
        if (lane == 0) store_wait_read();  // the slot's last store
        __syncwarp();
        if (add) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int r = 4 * q + (lane >> 3);
                *reinterpret_cast<float4*>(slot + r * 128 + 16 * ((lane ^ r) & 7)) = a.f[q];
            }
            __syncwarp();
            a.load(from + c + 64, p.C, p.J - n, cols - c - 64, lane);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float4* piece = reinterpret_cast<float4*>(at + 16 * (q ^ (lane & 7)));
            float4 f = make_float4(__uint_as_float(s.v[i][4 * q]), __uint_as_float(s.v[i][4 * q + 1]),
                                   __uint_as_float(s.v[i][4 * q + 2]), __uint_as_float(s.v[i][4 * q + 3]));
            if (add) {
                const float4 g = *piece;
                f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
            }
            *piece = f;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && n < p.J) {
            store_3d(tm_out, slot, t.k0 + c, n, t.e);
            store_commit();
        }
    }
}

// ---- the kernel ---------------------------------------------------------------------------
// tm_a: the M operand (weights; dy), tm_b: the N operand (rows; x). Gradient form: tm_ta and
// tm_tb are those in boxes of a unit, tm_out and tm_add the gradient and its addend.
template <int MODE, int ACT, int KIND>
__global__ void __launch_bounds__(Shape<MODE, KIND>::THREADS, 1)
ragged_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_ta, const __grid_constant__ CUtensorMap tm_tb,
              const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_add,
              const RaggedParams p) {
    using S = Shape<MODE, KIND>;
    constexpr bool RING = MODE == WGRAD && in_registers(KIND), CHUNKED = MODE == WGRAD && KIND != G16;
    constexpr int CHUNK = gradient_chunk(!in_16_bits(KIND), ACT);
    extern __shared__ __align__(1024) uint8_t smem[];
    Tail& s = *reinterpret_cast<Tail*>(smem + S::TAIL_AT);
    const WaitCtx wc{&s.abort_flag, p.err, p.wait_ns};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();  // 0: leader

    // set up while the kernel before this one ends; then its results may be read, and the next one may set up
    if (tid == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < TBUFS; ++i) {
            mbar_init(&s.tloc[i], 1);
            mbar_init(&s.tready[i], 2);
            mbar_init(&s.tfree[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 2 * S::WARPS);  // the pair's epilogue warps
        }
        for (int i = 0; i < 16; ++i) {
            mbar_init(&s.slot[i >> 2][i & 3], 1);
            mbar_init(&s.sdone[i >> 2][i & 3], 1);
        }
        mbar_init(&s.mma_done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        if (MODE == WGRAD) {
            tma_prefetch_desc(&tm_ta);
            tma_prefetch_desc(&tm_tb);
            tma_prefetch_desc(&tm_out);
            tma_prefetch_desc(&tm_add);
        }
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc_pair(&s.tmem_base, 512);
        tmem_relinquish_pair();
    }
    pdl_wait();
    pdl_launch_next();
    const int bad = build_tiles<MODE>(s, p);  // identical in both CTAs
    if (tid == 0 && bad && blockIdx.x == 0) set_err(p.err, MOE_DEV_ERR_OFFSETS);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers initialised, TMEM allocated
    tc_fence_after();
    const int n_tiles = s.n_tiles;
    const uint32_t tmem = s.tmem_base;
    const uint32_t lead_full = mapa_shared(smem_u32(&s.full[0]), 0);
    const uint32_t lead_tempty = mapa_shared(smem_u32(&s.tempty[0]), 0);
    const uint32_t lead_tready = mapa_shared(smem_u32(&s.tready[0]), 0);
    const int KB = (p.C + BK - 1) / BK;
    // whether this CTA's share of the N operand is two boxes of 64 columns
    const bool second = MODE == WGRAD && (p.kleast + (p.kmore > 0)) * p.kunit > 128;
    const uint32_t b_bytes = MODE == WGRAD ? (second ? OPER : OPER / 2) : p.maxu * 8 * 128;  // its bytes
    const uint32_t stage_bytes = OPER + b_bytes, stages = n_stages<MODE, KIND>(stage_bytes);
    // blocks of a tile; of a gradient, those that its whole units of 16 rows fill
    auto blocks_of = [&](const Tile& t) { return MODE == WGRAD ? (t.rows / 16 + 3) / 4 : KB; };
    auto chunks_of = [&](const Tile& t) { return CHUNKED ? max(1, (blocks_of(t) + CHUNK - 1) / CHUNK) : 1; };

    if (warp < 4) {
        if constexpr (RING) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_ROLES));
        if (warp == 0 || warp == 2) {
            // ---------------- copies: warp 0 the M operand, warp 2 the N operand ----------------
            const bool is_a = warp == 0;
            uint32_t stage = 0, phase = 0;
            long issued = 0;
            bool ok = true;
            for (Walk at(p); at.tile < n_tiles && ok; at.next()) {
                const Tile t = get_tile<MODE>(s, p, at.tile);
                const int nb = blocks_of(t);
                for (int b = 0; b < nb; ++b) {
                    if (!mbar_wait_warp(&s.empty[stage], phase ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (is_a && rank == 0) mbar_arrive_expect_tx(&s.full[stage], 2 * (OPER + b_bytes));
                        const uint32_t bar = lead_full + stage * 8;
                        uint8_t* dst = smem + stage * stage_bytes + (is_a ? 0 : OPER);
                        if (MODE == WGRAD) {
                            const int r = t.m0 + b * BK;
                            if (is_a) {
                                const int n = t.j0 + 128 * static_cast<int>(rank);
                                tma_load_2d_pair(dst, &tm_a, n, r, bar);
                                tma_load_2d_pair(dst + 8192, &tm_a, n + 64, r, bar);
                            } else {
                                // (two boxes may bring more than the share)
                                const int k = t.k0 + t.n / 2 * static_cast<int>(rank);
                                tma_load_2d_pair(dst, &tm_b, k, r, bar);
                                if (second) tma_load_2d_pair(dst + 8192, &tm_b, k + 64, r, bar);
                            }
                        } else {
                            const int c = b * BK;
                            if (!is_a) {
                                // (the box has maxu * 8 rows; the MMA reads n / 2 of them)
                                tma_load_2d_pair(dst, &tm_b, c, t.m0 + static_cast<int>(rank) * (t.n / 2), bar);
                            } else if (MODE == ROWS_FWD) {
                                load_3d_pair(dst, &tm_a, c, t.j0 + 128 * static_cast<int>(rank), t.e, bar);
                            } else {
                                const int j = t.j0 + 128 * static_cast<int>(rank);
                                load_3d_pair(dst, &tm_a, j, c, t.e, bar);
                                load_3d_pair(dst + 8192, &tm_a, j + 64, c, t.e, bar);
                            }
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (is_a && rank == 0) {  // let every copy land before either CTA may exit
                const long ring = stages, from = issued > ring ? issued - ring : 0;
                for (long j = from; j < issued; ++j)
                    mbar_drain(&s.full[j % ring], static_cast<uint32_t>((j / ring) & 1), kWaitLimitNs / 8);
            }
        } else if (warp == 1) {
            if (rank == 0) {
                // ---------------- MMAs (leader) ----------------
                const uint32_t major = MODE == WGRAD ? kMajorA | kMajorB : MODE == ROWS_BACK ? kMajorA : 0u;
                constexpr uint32_t STEP_K = 32 >> 4, STEP_MN = 2048 >> 4;  // 16 contraction indices on, in descriptor units
                constexpr uint32_t step_a = MODE == ROWS_FWD ? STEP_K : STEP_MN, step_b = MODE == WGRAD ? STEP_MN : STEP_K;
                uint32_t stage = 0, phase = 0, tails = 0, cur = 0, uses = 0;  // uses: bit a, uses of accumulator a, mod 2
                bool ok = true;
                Tile next{};
                Walk at(p);
                if (at.tile < n_tiles) next = get_tile<MODE>(s, p, at.tile);
                while (at.tile < n_tiles && ok) {
                    const Tile t = next;
                    const int nb = blocks_of(t), chunks = chunks_of(t);
                    const uint32_t idesc = f16_idesc(ACT, 256, t.n) | major;
                    for (int ch = 0; ch < chunks && ok; ++ch) {
                        const uint32_t acc = RING || ch == 0 ? cur : cur ^ 1u;  // (later chunks: the other one)
                        if (!mbar_wait_warp(&s.tempty[acc], (uses >> acc & 1u) ^ 1u, wc)) {
                            ok = false;
                            break;
                        }
                        uses ^= 1u << acc;
                        tc_fence_after();
                        const uint32_t d = tmem + acc * 256;
                        const int b0 = CHUNKED ? ch * CHUNK : 0, b1 = CHUNKED ? min(nb, b0 + CHUNK) : nb;
                        for (int b = b0; b < b1; ++b) {
                            if (!mbar_wait_warp(&s.full[stage], phase, wc)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint32_t at = smem_u32(smem + stage * stage_bytes);
                            const uint64_t ad = MODE == ROWS_FWD ? sw128_desc(at) : mn_desc(at);
                            const uint64_t bd = MODE == WGRAD ? mn_desc(at + OPER) : sw128_desc(at + OPER);
                            const int steps = MODE == WGRAD ? min(4, t.rows / 16 - 4 * b) : 4;
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < BK / 16; ++k)
                                    if (MODE != WGRAD || k < steps)
                                        tc_mma_pair(d, ad + k * step_a, bd + k * step_b, idesc, b > b0 || k > 0);
                                tc_commit_pair(&s.empty[stage], 0x3);
                            }
                            __syncwarp();
                            if (++stage == stages) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                        if (!ok) break;
                        if (MODE == WGRAD && ch + 1 == chunks && t.rows % 16 != 0) {
                            const uint32_t tb = tails % TBUFS;
                            if (!mbar_wait_warp(&s.tready[tb], (tails / TBUFS) & 1u, wc)) {
                                ok = false;
                                break;
                            }
                            ++tails;
                            tc_fence_after();
                            const uint32_t at = smem_u32(smem + S::TBUF_AT + tb * TBUF);
                            if (elect_one()) {
                                tc_mma_pair(d, mn_desc(at, UNIT), mn_desc(at + 2 * UNIT, UNIT), idesc, b1 > b0);
                                tc_commit_pair(&s.tfree[tb], 0x3);
                            }
                            __syncwarp();
                        }
                        if (elect_one()) tc_commit_pair(&s.tfull[acc], 0x3);
                        __syncwarp();
                        if (RING) cur ^= 1u;
                    }
                    // (found while the MMAs run: it would hold up the next tile's)
                    at.next();
                    if (ok && at.tile < n_tiles) next = get_tile<MODE>(s, p, at.tile);
                    if (!RING && chunks == 1) cur ^= 1u;
                }
                if (elect_one()) tc_commit_pair(&s.mma_done, 0x1);
                __syncwarp();
                mbar_drain(&s.mma_done, 0, kWaitLimitNs / 8);
            }
        } else if (warp == 3) {
            if (MODE == WGRAD) {
                // ---------------- tails ----------------
                uint32_t tails = 0;
                for (Walk at(p); at.tile < n_tiles; at.next()) {
                    const Tile t = get_tile<MODE>(s, p, at.tile);
                    const int left = t.rows % 16;
                    if (left == 0) continue;
                    const uint32_t tb = tails % TBUFS, ph = (tails / TBUFS) & 1u;
                    ++tails;
                    if (!mbar_wait_warp(&s.tfree[tb], ph ^ 1u, wc)) break;
                    uint8_t* buf = smem + S::TBUF_AT + tb * TBUF;
                    if (elect_one()) {
                        const int r = t.m0 + t.rows - left;
                        const int n = t.j0 + 128 * static_cast<int>(rank), k = t.k0 + t.n / 2 * static_cast<int>(rank);
                        mbar_arrive_expect_tx(&s.tloc[tb], 4 * UNIT);
                        tma_load_2d(buf, &tm_ta, n, r, &s.tloc[tb]);
                        tma_load_2d(buf + UNIT, &tm_ta, n + 64, r, &s.tloc[tb]);
                        tma_load_2d(buf + 2 * UNIT, &tm_tb, k, r, &s.tloc[tb]);
                        tma_load_2d(buf + 3 * UNIT, &tm_tb, k + 64, r, &s.tloc[tb]);
                    }
                    __syncwarp();
                    if (!mbar_wait_warp(&s.tloc[tb], ph, wc)) {
                        mbar_drain(&s.tloc[tb], ph, kWaitLimitNs / 8);
                        break;
                    }
                    // row r of 64 columns is the 128 bytes at 128 r (the swizzle moves bytes within them)
                    for (int i = lane; i < (16 - left) * 32; i += 32) {
                        const int r = left + (i >> 5), piece = i & 31;
                        *reinterpret_cast<uint4*>(buf + (piece >> 3) * UNIT + r * 128 + (piece & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) arrive_remote(lead_tready + tb * 8);
                    __syncwarp();
                }
            }
        }
    } else if (MODE == WGRAD && KIND == GADD && warp >= 8) {
        if constexpr (MODE == WGRAD && KIND == GADD) {
            // ---------------- copies of addends and gradients, for the epilogue warp of the same quarter ----------------
            const int q = warp & 3;
            copy_slots(s, p, &tm_out, &tm_add, smem + S::STG_AT + q * S::STG_WARP, q,
                       128 * static_cast<int>(rank) + 32 * q, n_tiles, lane, wc);
        }
    } else {
        // ---------------- epilogue ----------------
        if constexpr (RING) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_SUMS));
        const int q = warp & 3;  // TMEM lane quarter
        const int half = warp >= 8, ew = warp - 4;  // which of its two warps, and of all
        const int n_off = 128 * static_cast<int>(rank) + 32 * q;
        uint8_t* stg = smem + S::STG_AT + ew * S::STG_WARP;
        [[maybe_unused]] uint32_t used = 0;
        uint32_t cur = 0, uses = 0;
        auto wait_full = [&](uint32_t acc) {
            if (!mbar_wait_warp(&s.tfull[acc], uses >> acc & 1u, wc)) return false;
            uses ^= 1u << acc;
            tc_fence_after();
            return true;
        };
        auto release = [&](uint32_t acc) {
            if (lane != 0) return;
            if (rank == 0) mbar_arrive(&s.tempty[acc]);
            else arrive_remote(lead_tempty + acc * 8);
        };
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        if constexpr (RING) {
            for (Walk at(p); at.tile < n_tiles; at.next()) {
                const Tile t = get_tile<MODE>(s, p, at.tile);
                const int chunks = chunks_of(t), cols = tile_cols(p, t);
                if constexpr (KIND == G32ADD) prefetch_addend(p, t, n_off + lane, 32 * half, cols);
                RowSums v;
                v.clear();
                auto next = [&] {
                    tc_fence_before();
                    __syncwarp();
                    release(cur);
                    cur ^= 1u;
                };
                // (without addends the last chunk is added step by step beside the stores: 8192
                // rows of 8 groups, 4096 x 3584, 170 us and 174; with them that would hold its
                // accumulator too long, 284 us and 222)
                const int early = KIND == G32ADD ? chunks : chunks - 1;
                bool ok = true;
                for (int ch = 0; ch < early; ++ch) {
                    ok = wait_full(cur);
                    if (!ok) break;
                    if (t.rows > 0)
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // (past the tile's columns too)
                            v.add(i, lanes + cur * 256 + 32 * half + 64 * i);
                    next();
                }
                if (KIND == G32) ok = ok && wait_full(cur);
                if (!ok) break;
                store_sums<KIND>(p, &tm_out, stg, v, lanes + cur * 256 + 32 * half, t, n_off, half, cols, lane);
                if (KIND == G32) next();
            }
        } else {
            for (Walk at(p); at.tile < n_tiles; at.next()) {
                const Tile t = get_tile<MODE>(s, p, at.tile);
                const int chunks = chunks_of(t);
                if constexpr (KIND == FULL) prefetch_residual(p, lane, t.m0, t.rows, t.j0 + n_off);
                if (!wait_full(cur)) break;
                const uint32_t ta = lanes + cur * 256, tb = lanes + (cur ^ 1u) * 256;
                bool ok = true;
                if constexpr (CHUNKED) {
                    for (int ch = 1; ch < chunks && ok; ++ch) {
                        ok = wait_full(cur ^ 1u);
                        if (ok && ch + 1 < chunks) {
                            fold<Slots<KIND>::COLS, S::HALVES>(ta, tb, half);
                            tc_fence_before();
                            __syncwarp();
                            release(cur ^ 1u);
                        }
                    }
                }
                if (!ok) break;
                if constexpr (MODE == WGRAD) {
                    if (!wgrad_epilogue<ACT, KIND>(s, p, &tm_out, stg, used, ta, tb, t.rows == 0 ? 0 : chunks > 1 ? 2 : 1, t,
                                                   ew, n_off, half, lane, wc))
                        break;
                } else {
                    rows_epilogue<ACT, KIND>(p, ta, smem_u32(stg), t, t.j0 + n_off, half, lane);
                }
                tc_fence_before();
                __syncwarp();
                release(cur);
                if (chunks > 1) release(cur ^ 1u);
                else cur ^= 1u;
            }
        }
        if (MODE == WGRAD && KIND != GADD && lane == 0) store_wait();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (s.abort_flag) {
        // a wait gave up: copies that the other CTA signals, or has signalled here, may still be on their way
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000) __nanosleep(1000);
    }
    __syncthreads();
    cluster_sync_all();  // the leader's MMAs read the peer's shared memory and write its TMEM
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---- launch -----------------------------------------------------------------------------

struct Maps {
    CUtensorMap a, b, ta, tb, out, add;
};

template <int MODE, int ACT, int KIND>
int launch(const Maps& m, const RaggedParams& p, int64_t tiles, cudaStream_t st, const char* who) {
    auto kernel = ragged_kernel<MODE, ACT, KIND>;
    constexpr int smem = Shape<MODE, KIND>::SMEM;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(Shape<MODE, KIND>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static PerDevice pairs;
    std::atomic<int>* known = pairs.here();
    int max_pairs = known ? known->load(std::memory_order_acquire) : 0;
    if (max_pairs == 0) {
        const int rc = set_smem_limit(reinterpret_cast<const void*>(kernel), smem);
        if (rc != MOE_OK) return rc;
        if (MODE == WGRAD && in_registers(KIND)) {  // (a larger share than the launch's would be waited for without end)
            cudaFuncAttributes fa;
            const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
            if (e != cudaSuccess || fa.numRegs < Shape<MODE, KIND>::REGS_LAUNCH)
                return fail(MOE_ERR_CUDA, "%s: the kernel was built with too few registers", who);
        }
        const int sms = sm_count();
        cfg.gridDim = dim3(sms > 1 ? sms / 2 * 2 : 2);
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&max_pairs, kernel, &cfg);
        if (e != cudaSuccess || max_pairs <= 0)
            return fail(MOE_ERR_CUDA, "%s: cannot place pairs of CTAs: %s", who, cudaGetErrorString(e));
        if (known) known->store(max_pairs, std::memory_order_release);
    }
    if (tiles > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
    const int pairs_used = static_cast<int>(tiles < max_pairs ? tiles : max_pairs);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs_used));
    RaggedParams q = p;
    if (MODE == WGRAD && tiles > max_pairs)
        while (q.turn + 1 < pairs_used && std::gcd(static_cast<unsigned>(pairs_used + q.turn), p.per.d) != 1) ++q.turn;
    cfg.stream = st;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, m.ta, m.tb, m.out, m.add, q);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

template <int MODE, int ACT> int launch_rows_form(const RaggedArgs& g, int maxu) {
    RaggedParams p = g.p;
    p.maxu = maxu;
    p.units.set(maxu);
    Maps m;
    // tall tiles are bound by what comes from L2, low ones by the weights' way from HBM
    const bool reused = p.maxu >= 8;
    int rc = make_tmap_3d(&m.a, const_cast<void*>(g.w), g.act, g.K, g.N, p.E, 64, MODE == ROWS_FWD ? 128 : 64, reused);
    if (rc == MOE_OK) rc = make_tmap_2d(&m.b, g.a, p.rows, p.C, p.maxu * 8, g.act, reused);
    if (rc != MOE_OK) return rc;
    m.ta = m.tb = m.out = m.add = m.b;
    // row tiles at most: one more per group than the rows fill
    const int64_t row_tiles = (p.rows + 16 * p.maxu - 1) / (16 * p.maxu) + (p.E > 1 ? p.E : 0);
    const int64_t tiles = row_tiles * ((p.J + 255) / 256);
    if (MODE == ROWS_FWD && (p.bias || p.residual || p.pre || p.fn != MOE_FN_NONE))
        return launch<ROWS_FWD, ACT, FULL>(m, p, tiles, g.st, g.who);
    return launch<MODE, ACT, PLAIN>(m, p, tiles, g.st, g.who);
}

}  // namespace
}  // namespace ragged
}  // namespace moe
