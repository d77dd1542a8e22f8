// E4M3 matrix product with block scales on the 5th-generation tensor cores,
// for more rows than the streaming form (block_fp8.cu) takes.
//
//     out[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in b} a[m, k] w[n, k]  (+ addend[m, n])
//
// The scales are any f32 values, so they cannot ride in the MMA: each block of
// 128 contraction indices is one accumulation group (four tcgen05.mma of K =
// 32) into a fresh TMEM buffer, and the epilogue warps read every buffer
// back, multiply by sa * sb and add to f32 sums in registers. Rows of a are
// TMEM lanes, so sa is one value per thread and block, and a warp's columns
// lie in one block of 128 weight rows, so sb is one value per warp. Where a
// lane's sa * sb lies outside [2^-63, 2^65), the warp multiplies twice
// (scale_before; rows of zeros, whose scale is 2^-126, among others: M = 4096,
// N = 28672, K = 4096 434 us with half the rows zeros, 373 with none). The
// buffers are a ring: the MMAs of the next blocks run while one is read back.
//   * 128 x BN tiles, BN = 256 when that fills the GPU. What limits it is the
//     round trip of a buffer (MMAs, the signal, reading it back, the signal
//     back) against the two buffers that 512 TMEM columns hold. So a buffer is
//     read back by many warps at once, 64 columns each, and nothing else
//     stands in their way: a warp fetches the scales of a block while its MMAs
//     run and leaves them in shared memory. A thread needs about 650 clocks to
//     wait for, issue and commit a block's MMAs, whatever their width, so two
//     threads issue, a block each in turn (their buffers are independent).
//     CTA pairs (M = 256) halve the shared-memory traffic but lengthen every
//     signal by a cluster hop, and measured slower.
//   * Too few tiles for the GPU: a cluster of 2 or 4 CTAs per tile, each with a
//     part of the contraction; each CTA then adds a slice of the columns, in
//     rank order, from all of them (distributed shared memory).
//   * Finished rows leave through a staging area by TMA stores.
//   * Roles: warp 0 copies (TMA, 128-byte swizzle), warps 1 and 2 issue the
//     MMAs, warp 3 fetches scales, the others add and store. Every wait is
//     bounded. At BN = 256 the 20 warps' 96 registers are split 32 / 112
//     between the first four and the others. (A second copying warp, and
//     scales fetched two blocks ahead, measured 5 to 10% slower; a second
//     staging area, in the place of the fourth stage, the same.)
// Measured: M = 4096, N = 28672, K = 4096 373 us (2.58 PFLOP/s; 415 in long runs,
// at lower clocks; tensor pipe 55% busy: 465 ns a block of 128 x 256 x 128, of which
// its MMAs take half, and 1.5 us a tile for the stores); M = 17, N = 4096,
// K = 14336 16.3 us (8.7 for the bytes: 28 blocks at 5.5 TB/s and the meeting of
// four CTAs).
#include "block_fp8.cuh"
#include "tc_ring.cuh"

namespace moe {
namespace {

constexpr int kTcA = 128 * 128;  // bytes of a stage's activation rows per CTA

template <int BN, int PARTS> struct TcShape {
    static constexpr int STAGE = kTcA + BN * 128;
    static constexpr int STAGES = tc_stages(BN), NBUF = tc_buffers(BN);
    static_assert(STAGES % kTcIssuers == 0 && NBUF % kTcIssuers == 0, "every stage and buffer is one issuing thread's");
    static constexpr int COLS = NBUF * BN;             // TMEM columns
    static constexpr int GROUPS = BN == 64 ? 2 : 4;    // warpgroups that read a buffer back
    static constexpr int EPI_WARPS = 4 * GROUPS, THREADS = 128 + 128 * GROUPS;
    static constexpr int PER = BN / GROUPS;            // columns per epilogue warp
    static constexpr int OUT_BYTES = PARTS > 1 ? 0 : 32 * 32 * 2;   // a warp's staging area: 32 x 32 outputs
    static constexpr int OUT_AT = STAGES * STAGE;
    static constexpr int SCALE_AT = OUT_AT + EPI_WARPS * OUT_BYTES; // [NBUF]: 128 row scales, 2 column block scales
    static constexpr int SCALES = 136;                              // floats of a buffer's scales
    static constexpr int TAIL_AT = SCALE_AT + NBUF * SCALES * 4;
    static constexpr int SMEM = TAIL_AT + 256;  // (nothing to align by hand: the array is declared aligned)
    static_assert(SMEM <= 232448, "shared memory over the limit");
};

struct TcTail {
    uint64_t full[8], empty[8], tfull[4], tempty[4], mma_done[kTcIssuers];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(TcTail) <= 256, "tail");

// kind::f8f6f4 with f32 accumulation, E4M3 x E4M3, both K-major: D format f32
// (bits 4-5 = 1), A and B format E4M3 (0), N >> 3 (17-22), M >> 4 (24-28)
__host__ __device__ constexpr uint32_t e4m3_idesc(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// shared memory -> global through the tensor map (rows and columns past its
// bounds are not written), in this thread's bulk group
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// this thread's bulk stores have read their shared memory
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// ... and are complete
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// (lo, hi) += (s, s) * (a, b), each rounded once
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t s2, uint32_t a, uint32_t b) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %3};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}"
        : "+l"(acc)
        : "l"(s2), "r"(a), "r"(b));
}

// (a, b) *= (s, s)
__device__ __forceinline__ void mul2(uint32_t& a, uint32_t& b, float s) {
    asm("{\n\t.reg .b64 v, t;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 t, {%2, %2};\n\tmul.rn.f32x2 v, v, t;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+r"(a), "+r"(b)
        : "f"(s));
}

template <int N> __device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct TcTile {
    int m0, n0;
};
// Tiles in groups of up to 16 row tiles: all rows of a group for one column
// tile, then the next, so a wave of CTAs shares few weight tiles and the
// group's activations stay in L2.
template <int BN> __device__ __forceinline__ TcTile tc_tile(const BfParams& p, int t) {
    const int mt = (p.M + 127) / 128, ntl = (p.N + BN - 1) / BN;
    const int per = 16 * ntl, grp = t / per, in = t - grp * per;
    const int rows = min(16, mt - 16 * grp);
    return {(16 * grp + in % rows) * 128, in / rows * BN};
}

// PARTS > 1: one tile per cluster of PARTS CTAs; otherwise one CTA walks tiles.
template <int ACT, int BN, int PARTS>
__global__ void __launch_bounds__(TcShape<BN, PARTS>::THREADS, 1)
block_fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_o, const BfParams p, int a_rows, int32_t* err, uint64_t wait_ns) {
    using S = TcShape<BN, PARTS>;
    pdl_wait();
    // The array is aligned, so the offset is 0. It is computed all the same: with a base
    // that the compiler knows, the narrow tiles measured 2 to 5% slower.
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint32_t base;
    asm("mov.u32 %0, %1;" : "=r"(base) : "r"(smem_u32(smem_raw)));
    uint8_t* smem = smem_raw + ((1024u - (base & 1023u)) & 1023u);
    TcTail& s = *reinterpret_cast<TcTail*>(smem + S::TAIL_AT);
    const WaitCtx wc{&s.abort_flag, err, wait_ns};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr bool SPLIT = PARTS > 1;
    const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = blockIdx.x / PARTS, step = SPLIT ? 1 << 30 : gridDim.x;
    // this CTA's contraction blocks
    const int kb0 = p.kb * rank / PARTS, kbs = p.kb * (rank + 1) / PARTS - kb0;
    const int n_tiles = ((p.M + 127) / 128) * ((p.N + BN - 1) / BN);

    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < S::NBUF; ++i) {
            mbar_init(&s.tfull[i], 2);  // the MMAs, and its scales
            mbar_init(&s.tempty[i], S::EPI_WARPS);
        }
        for (int i = 0; i < kTcIssuers; ++i) mbar_init(&s.mma_done[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == 1) {
        tmem_alloc(&s.tmem_base, S::COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_o);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;

    if (warp < 4) {
        if (BN == 256) regs_dec<32>();  // 4 x 32 + 16 x 112 = 20 x 96
        if (warp == 0 && lane == 0) {
            // ---------------- copies ----------------
            const uint32_t bytes = a_rows * 128 + BN * 128;
            uint32_t stage = 0, phase = 0;
            long issued = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                const TcTile t = tc_tile<BN>(p, tile);
                for (int b = kb0; b < kb0 + kbs; ++b) {
                    if (!mbar_wait(&s.empty[stage], phase ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&s.full[stage], bytes);
                    uint8_t* dst = smem + stage * S::STAGE;
                    tma_load_2d(dst, &tm_a, b * 128, t.m0, &s.full[stage]);
                    tma_load_2d(dst + kTcA, &tm_w, b * 128, t.n0, &s.full[stage]);
                    ++issued;
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // let every copy land before the CTA may exit
            const long from = issued > S::STAGES ? issued - S::STAGES : 0;
            for (long j = from; j < issued; ++j)
                mbar_drain(&s.full[j % S::STAGES], static_cast<uint32_t>((j / S::STAGES) & 1), kWaitLimitNs / 8);
        } else if ((warp == 1 || warp == 2) && lane == 0) {
            // ---------------- MMAs: one accumulation group per block, every other block ----------------
            constexpr uint32_t idesc = e4m3_idesc(128, BN);
            const int64_t mine = first < n_tiles ? (n_tiles - 1 - first) / step + 1 : 0;
            const int64_t blocks = mine * kbs;
            // block i: stage i mod STAGES, buffer i mod NBUF, and their phases. Both are this
            // thread's alone (tc_ring.cuh): a wait by parity needs the phase before to have been seen
            uint32_t stage = warp - 1, phase = 0, buf = warp - 1, bphase = 0;
            bool ok = warp - 1 < blocks && mbar_wait(&s.full[stage], 0, wc);
            for (int64_t i = warp - 1; i < blocks && ok; i += kTcIssuers) {
                if (!mbar_wait(&s.tempty[buf], bphase ^ 1, wc)) break;
                tc_fence_after();
                const uint64_t ad = sw128_desc(smem_u32(smem + stage * S::STAGE));
                const uint64_t bd = sw128_desc(smem_u32(smem + stage * S::STAGE + kTcA));
                const uint32_t d = tmem + buf * BN, at = stage;
                mma_e4m3(d, ad, bd, idesc, 0);
                mma_e4m3(d, ad + 2, bd + 2, idesc, 1);
                mma_e4m3(d, ad + 4, bd + 4, idesc, 1);
                mma_e4m3(d, ad + 6, bd + 6, idesc, 1);
                tc_commit(&s.tfull[buf]);
                tc_commit(&s.empty[at]);
                stage += kTcIssuers;
                if (stage >= S::STAGES) {
                    stage -= S::STAGES;
                    phase ^= 1;
                }
                buf += kTcIssuers;
                if (buf >= S::NBUF) {
                    buf -= S::NBUF;
                    bphase ^= 1;
                }
                if (i + kTcIssuers < blocks) ok = mbar_wait(&s.full[stage], phase, wc);
            }
            tc_commit(&s.mma_done[warp - 1]);
            mbar_drain(&s.mma_done[warp - 1], 0, kWaitLimitNs / 8);
        } else if (warp == 3) {
            // ---------------- scales: four rows a lane ----------------
            float* scales = reinterpret_cast<float*>(smem + S::SCALE_AT);
            uint32_t buf = 0, bphase = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                const TcTile t = tc_tile<BN>(p, tile);
                const float* sa[4];
                float a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sa[j] = p.sa + static_cast<size_t>(min(t.m0 + 4 * lane + j, p.M - 1)) * p.kb + kb0;
                    a[j] = __ldg(sa[j]);
                }
                // lanes 0 and 1: the scales of the tile's first and second 128 columns
                const float* sb =
                    p.sb + static_cast<size_t>(min(t.n0 + 128 * (lane & 1), p.N - 1) / kQuantGroup) * p.kb + kb0;
                float b0 = __ldg(sb);
                for (int b = 0; b < kbs; ++b) {
                    const float4 v = make_float4(a[0], a[1], a[2], a[3]);
                    const float vb = b0;
                    const int nb = min(b + 1, kbs - 1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = __ldg(sa[j] + nb);
                    b0 = __ldg(sb + nb);
                    if (!mbar_wait_warp(&s.tempty[buf], bphase ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    float* dst = scales + buf * S::SCALES;
                    *reinterpret_cast<float4*>(dst + 4 * lane) = v;
                    if (lane < 2) dst[128 + lane] = vb;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.tfull[buf]);
                    if (++buf == S::NBUF) {
                        buf = 0;
                        bphase ^= 1;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        if (BN == 256) regs_inc<112>();
        // ---------------- scale, add, store ----------------
        const int q = warp & 3, grp = (warp - 4) >> 2;
        const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + grp * S::PER;
        const float* scales = reinterpret_cast<const float*>(smem + S::SCALE_AT);
        uint8_t* out = smem + S::OUT_AT + (warp - 4) * S::OUT_BYTES;
        uint32_t buf = 0, bphase = 0;
        bool ok = true;
        for (int tile = first; tile < n_tiles && ok; tile += step) {
            uint64_t acc[S::PER / 2];
#pragma unroll
            for (int j = 0; j < S::PER / 2; ++j) acc[j] = 0;
            for (int b = 0; b < kbs; ++b) {
                if (!mbar_wait_warp(&s.tfull[buf], bphase, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float sa = scales[buf * S::SCALES + 32 * q + lane];
                const float sb = scales[buf * S::SCALES + 128 + (BN == 256 ? grp / 2 : 0)];
                float sc = sa * sb;
                // of the warp, since the branch on it lies between warp-wide TMEM loads
                const bool odd = __any_sync(0xffffffffu, !scale_ordinary(sc));
                const float before = odd ? scale_before(sc, sa, sb) : 1.0f;
                uint64_t s2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(sc));
#pragma unroll
                for (int c = 0; c < S::PER; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(ta + buf * BN + c, r);
                    tmem_ld_wait_regs(r);
                    if (c + 32 == S::PER) {  // the buffer is read: the MMAs of a later block may have it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s.tempty[buf]);
                    }
                    if (odd)
#pragma unroll
                        for (int j = 0; j < 16; ++j) mul2(r[2 * j], r[2 * j + 1], before);
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[c / 2 + j], s2, r[2 * j], r[2 * j + 1]);
                }
                if (++buf == S::NBUF) {
                    buf = 0;
                    bphase ^= 1;
                }
            }
            if (SPLIT) {
                // the stages are free once every CTA of the cluster is done with its products
                __syncwarp();
                cluster_sync_all();
                // 16 bytes (four columns) of every thread, by source CTA and piece of the slice
                constexpr int SLICE = S::PER / PARTS, PIECES = SLICE / 4, PLANE = S::EPI_WARPS * 32 * 16;
                uint8_t* sums = smem + ((warp - 4) * 32 + lane) * 16;
#pragma unroll
                for (int r = 0; r < PARTS; ++r) {
                    const uint32_t to = mapa_shared(smem_u32(sums + rank * PIECES * PLANE), r);
#pragma unroll
                    for (int j = 0; j < PIECES; ++j)
                        asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(to + j * PLANE),
                                     "l"(acc[(r * SLICE + 4 * j) / 2]), "l"(acc[(r * SLICE + 4 * j) / 2 + 1])
                                     : "memory");
                }
                __syncwarp();
                cluster_sync_all();
                const TcTile t = tc_tile<BN>(p, tile);
                const int m = t.m0 + 32 * q + lane, n = t.n0 + grp * S::PER + rank * SLICE;
                if (!ok || m >= p.M) break;
                const size_t at = static_cast<size_t>(m) * p.N + n;
#pragma unroll
                for (int c = 0; c < SLICE; c += 8) {
                    if (n + c >= p.N) break;
                    float v[8];
#pragma unroll
                    for (int r = 0; r < PARTS; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 f =
                                *reinterpret_cast<const float4*>(sums + (r * PIECES + c / 4 + h) * PLANE);
                            v[4 * h] = r ? v[4 * h] + f.x : f.x;
                            v[4 * h + 1] = r ? v[4 * h + 1] + f.y : f.y;
                            v[4 * h + 2] = r ? v[4 * h + 2] + f.z : f.z;
                            v[4 * h + 3] = r ? v[4 * h + 3] + f.w : f.w;
                        }
                    if (p.addend) {
                        float f[8];
                        unpack8<ACT>(*reinterpret_cast<const uint4*>(p.addend + at + c), f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += f[j];
                    }
                    *reinterpret_cast<uint4*>(p.out + at + c) = pack8<ACT>(v);
                }
                break;
            }
            if (!ok) break;
            // through the staging area, whose 16-byte pieces lie swizzled by row as the
            // store's tensor map expects
            const TcTile t = tc_tile<BN>(p, tile);
            const int m = t.m0 + 32 * q + lane, n = t.n0 + grp * S::PER;
            const bool row = m < p.M;
            const size_t at = static_cast<size_t>(m) * p.N + n;
#pragma unroll
            for (int c0 = 0; c0 < S::PER; c0 += 32) {
                if (n + c0 >= p.N) break;
                if (lane == 0) bulk_wait_read();  // the area's last store
                __syncwarp();
#pragma unroll
                for (int c = c0; c < c0 + 32; c += 8) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t w = acc[c / 2 + j];
                        v[2 * j] = __uint_as_float(static_cast<uint32_t>(w));
                        v[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(w >> 32));
                    }
                    if (p.addend && row && n + c < p.N) {
                        float f[8];
                        unpack8<ACT>(*reinterpret_cast<const uint4*>(p.addend + at + c), f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += f[j];
                    }
                    const int piece = ((c - c0) / 8) ^ ((lane >> 1) & 3);
                    *reinterpret_cast<uint4*>(out + lane * 64 + 16 * piece) = pack8<ACT>(v);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && t.m0 + 32 * q < p.M) {
                    tma_store_2d(&tm_o, out, n + c0, t.m0 + 32 * q);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait();
    }

    if (SPLIT && warp < 4) {  // the other warps' two meetings
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, S::COLS);
}

template <int ACT, int BN, int PARTS>
int launch_tc(const BfParams& p, int sms, int32_t* err, cudaStream_t st, const char* who) {
    using S = TcShape<BN, PARTS>;
    static_assert(PARTS == 1 || S::EPI_WARPS * 32 * S::PER * 4 <= S::OUT_AT, "a tile's sums fit in the stages");
    auto kernel = block_fp8_tc_kernel<ACT, BN, PARTS>;
    static int configured_for = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        const int rc = set_smem_limit(reinterpret_cast<const void*>(kernel), S::SMEM);
        if (rc != MOE_OK) return rc;
        configured_for = dev;
    }
    CUtensorMap tm_a, tm_w, tm_o;
    // of few rows, no more are copied than there may be (the other TMEM lanes hold sums nobody reads)
    const int a_rows = p.M >= 128 ? 128 : (p.M + 15) / 16 * 16;
    int rc = make_tmap_2d_u8(&tm_a, p.a, p.M, p.K, a_rows);
    if (rc == MOE_OK) rc = make_tmap_2d_u8(&tm_w, p.w, p.N, p.K, BN);
    if (rc == MOE_OK) rc = make_tmap_2d_out(&tm_o, p.out, p.M, p.N, 32, 32, ACT);
    if (rc != MOE_OK) return rc;
    const int64_t tiles = static_cast<int64_t>((p.M + 127) / 128) * ((p.N + BN - 1) / BN);
    if (tiles > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "%s: M=%d x N=%d is too large", who, p.M, p.N);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = PARTS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(PARTS > 1 ? tiles * PARTS : (tiles < sms ? tiles : sms)));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = PARTS > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_w, tm_o, p, a_rows, err, wait_limit_ns());
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

// Tile width and split of the contraction, by the time that each choice would
// take: the waves of CTAs, times the blocks of 128 of each at what a block
// costs at that width (260, 315 and 465 ns at 64, 128 and 256 columns) and what
// a tile's end holds up the next (0.3, 0.7 and 1.5 us), and what a launch costs
// (2.5 us; 4.5 and 5.5 with the meeting of 2 or 4 CTAs). The costs are fitted to
// 96 sizes measured on a GB300 at every form: the choice is 0.4% slower than the
// best form in the mean. A wide tile reads less and spends fewer steps per sum,
// a narrow or split one fills more of the GPU: M = 128, N = 4096, K = 14336 takes
// 16.6 us at 128 x 4 CTAs, 19.4 at 64 x 2, 31 at 64 and 56 at 256; M = 2048,
// N = 2816, K = 2048 20.4 at 256, 19.9 at 128, 24.1 at 64. A tile is split only
// where every CTA runs at once: each wave of clusters begins and ends anew, and
// those 352 tiles took 36 us at 128 x 2.
template <int ACT> int pick_tc(const BfParams& p, int sms, int32_t* err, cudaStream_t st, const char* who) {
    static const struct {
        int bn, parts, block_ns, tile_ns, fixed_ns;
    } forms[] = {{256, 1, 465, 1500, 2500}, {128, 1, 315, 700, 2500}, {64, 1, 260, 300, 2500}, {128, 2, 315, 0, 4500},
                 {64, 2, 260, 0, 4500},     {128, 4, 315, 0, 5500},   {64, 4, 260, 0, 5500}};
    int best = 0;
    int64_t best_ns = INT64_MAX;
    for (int i = 0; i < 7; ++i) {
        const auto& f = forms[i];
        const int64_t ctas = static_cast<int64_t>((p.M + 127) / 128) * ((p.N + f.bn - 1) / f.bn) * f.parts;
        if (f.parts > 1 && (p.kb < f.parts || ctas > sms)) continue;
        const int64_t blocks = (p.kb + f.parts - 1) / f.parts;
        const int64_t ns = (ctas + sms - 1) / sms * (blocks * f.block_ns + f.tile_ns) + f.fixed_ns;
        if (ns < best_ns) {
            best_ns = ns;
            best = i;
        }
    }
    switch (best) {
        case 0: return launch_tc<ACT, 256, 1>(p, sms, err, st, who);
        case 1: return launch_tc<ACT, 128, 1>(p, sms, err, st, who);
        case 2: return launch_tc<ACT, 64, 1>(p, sms, err, st, who);
        case 3: return launch_tc<ACT, 128, 2>(p, sms, err, st, who);
        case 4: return launch_tc<ACT, 64, 2>(p, sms, err, st, who);
        case 5: return launch_tc<ACT, 128, 4>(p, sms, err, st, who);
        default: return launch_tc<ACT, 64, 4>(p, sms, err, st, who);
    }
}

}  // namespace

int launch_block_fp8_tc(const BfParams& p, int act, int sms, int32_t* err, cudaStream_t st, const char* who) {
    return act == MOE_ACT_BF16 ? pick_tc<MOE_ACT_BF16>(p, sms, err, st, who)
                               : pick_tc<MOE_ACT_F16>(p, sms, err, st, who);
}

}  // namespace moe
