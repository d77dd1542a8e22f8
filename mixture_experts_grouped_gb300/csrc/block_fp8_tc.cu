// E4M3 matrix product with block scales on the 5th-generation tensor cores,
// for more rows than the streaming form (block_fp8.cu) takes.
//
//     out[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in b} a[m, k] w[n, k]  (+ addend[m, n])
//
// The scales are any f32 values, so they cannot ride in the MMA: each block of
// 128 contraction indices is one accumulation group (four tcgen05.mma of K =
// 32) into a fresh TMEM buffer, and eight epilogue warps read every buffer
// back, multiply by sa * sb and add to f32 sums in registers. Rows of a are
// TMEM lanes, so sa is one value per thread and block, and a warp's columns
// lie in one block of 128 weight rows, so sb is one value per warp. The
// buffers are a ring: the MMAs of the next blocks run while one is read back.
//   * BN columns per tile, 128 rows per CTA; CG = 2: a CTA pair
//     (tcgen05.mma.cta_group::2, M = 256, each CTA holding half of the tile's
//     weight rows), which halves the shared-memory traffic per MMA.
//   * Cost per block and CTA at BN = 256: 512 clocks of MMA; 128 x 256 sums
//     read from TMEM and 16384 packed f32 FMAs (128 clocks), so the
//     scaling hides behind the MMAs.
//   * Roles: warp 0 copies (TMA, 128-byte swizzle), warp 1 issues the MMAs,
//     warps 4-11 scale, add and store. Every wait is bounded. At BN = 256 the
//     sums alone are 128 registers a thread, so the launch's 12 x 168 registers
//     are split 88 / 208 between the first warpgroup and the others.
#include "block_fp8.cuh"

namespace moe {
namespace {

constexpr int kTcThreads = 384;   // warpgroup 0: copies, MMAs (and two idle warps); 1 and 2: scale, add, store
constexpr int kTcEpiWarps = 8;
constexpr int kTcA = 128 * 128;  // bytes of a stage's activation rows per CTA

template <int CG, int BN> struct TcShape {
    static constexpr int B_ROWS = BN / CG;             // weight rows per CTA and stage
    static constexpr int STAGE = kTcA + B_ROWS * 128;
    static constexpr int STAGES = 196608 / STAGE < 8 ? 196608 / STAGE : 8;
    static constexpr int NBUF = 512 / BN < 4 ? 512 / BN : 4;
    static constexpr int COLS = NBUF * BN;             // TMEM columns
    static constexpr int HALF = BN / 2;                // columns per epilogue warp
    static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
};

struct TcTail {
    uint64_t full[8], empty[8], tfull[4], tempty[4], mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(TcTail) <= 256, "tail");

// kind::f8f6f4 with f32 accumulation, E4M3 x E4M3, both K-major: D format f32
// (bits 4-5 = 1), A and B format E4M3 (0), N >> 3 (17-22), M >> 4 (24-28)
__host__ __device__ constexpr uint32_t e4m3_idesc(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// (lo, hi) += (s, s) * (a, b), each rounded once
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t s2, uint32_t a, uint32_t b) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %3};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}"
        : "+l"(acc)
        : "l"(s2), "r"(a), "r"(b));
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
template <int CG, int BN> __device__ __forceinline__ TcTile tc_tile(const BfParams& p, int t) {
    const int mt = (p.M + 128 * CG - 1) / (128 * CG), ntl = (p.N + BN - 1) / BN;
    const int per = 16 * ntl, grp = t / per, in = t - grp * per;
    const int rows = min(16, mt - 16 * grp);
    return {(16 * grp + in % rows) * 128 * CG, in / rows * BN};
}

template <int ACT, int CG, int BN>
__global__ void __launch_bounds__(kTcThreads, 1)
block_fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                    const BfParams p, int32_t* err, uint64_t wait_ns) {
    using S = TcShape<CG, BN>;
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    TcTail& s = *reinterpret_cast<TcTail*>(smem + S::STAGES * S::STAGE);
    const WaitCtx wc{&s.abort_flag, err, wait_ns};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int n_tiles = ((p.M + 128 * CG - 1) / (128 * CG)) * ((p.N + BN - 1) / BN);

    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < S::NBUF; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], CG * kTcEpiWarps);
        }
        mbar_init(&s.mma_done, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == 1) {
        if (CG == 2) {
            tmem_alloc_pair(&s.tmem_base, S::COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&s.tmem_base, S::COLS);
            tmem_relinquish();
        }
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_w);
    }
    tc_fence_before();
    if (CG == 2) cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;

    if (warp < 4) {
        if (BN == 256) regs_dec<88>();  // 4 x 88 + 8 x 208 = 12 x 168
        if (warp == 0 && lane == 0) {
            // ---------------- copies ----------------
            const uint32_t full0 = CG == 2 ? mapa_shared(smem_u32(&s.full[0]), 0) : 0;
            uint32_t stage = 0, phase = 0;
            long issued = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                const TcTile t = tc_tile<CG, BN>(p, tile);
                const int arow = t.m0 + 128 * static_cast<int>(rank);
                const int wrow = t.n0 + S::B_ROWS * static_cast<int>(rank);
                for (int b = 0; b < p.kb; ++b) {
                    if (!mbar_wait(&s.empty[stage], phase ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], CG * S::STAGE);
                    uint8_t* dst = smem + stage * S::STAGE;
                    if (CG == 2) {
                        tma_load_2d_pair(dst, &tm_a, b * 128, arow, full0 + stage * 8);
                        tma_load_2d_pair(dst + kTcA, &tm_w, b * 128, wrow, full0 + stage * 8);
                    } else {
                        tma_load_2d(dst, &tm_a, b * 128, arow, &s.full[stage]);
                        tma_load_2d(dst + kTcA, &tm_w, b * 128, wrow, &s.full[stage]);
                    }
                    ++issued;
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (rank == 0) {  // let every copy land before the CTA (or either of the pair) may exit
                const long from = issued > S::STAGES ? issued - S::STAGES : 0;
                for (long j = from; j < issued; ++j)
                    mbar_drain(&s.full[j % S::STAGES], static_cast<uint32_t>((j / S::STAGES) & 1), kWaitLimitNs / 8);
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---------------- MMAs: one accumulation group per block ----------------
            constexpr uint32_t idesc = e4m3_idesc(128 * CG, BN);
            uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += step) {
                for (int b = 0; b < p.kb; ++b) {
                    if (!mbar_wait(&s.tempty[buf], bphase ^ 1, wc) || !mbar_wait(&s.full[stage], phase, wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = sw128_desc(smem_u32(smem + stage * S::STAGE));
                    const uint64_t bd = sw128_desc(smem_u32(smem + stage * S::STAGE + kTcA));
                    const uint32_t d = tmem + buf * BN;
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_e4m3<CG>(d, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                    if (CG == 2) {
                        tc_commit_pair(&s.empty[stage], 0x3);
                        tc_commit_pair(&s.tfull[buf], 0x3);
                    } else {
                        tc_commit(&s.empty[stage]);
                        tc_commit(&s.tfull[buf]);
                    }
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                    if (++buf == S::NBUF) {
                        buf = 0;
                        bphase ^= 1;
                    }
                }
            }
            if (CG == 2) tc_commit_pair(&s.mma_done, 0x1);
            else tc_commit(&s.mma_done);
            mbar_drain(&s.mma_done, 0, kWaitLimitNs / 8);
        }
        __syncwarp();
    } else {
        if (BN == 256) regs_inc<208>();
        // ---------------- scale, add, store ----------------
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * S::HALF;
        const uint32_t tempty0 = CG == 2 ? mapa_shared(smem_u32(&s.tempty[0]), 0) : 0;
        uint32_t buf = 0, bphase = 0;
        bool ok = true;
        for (int tile = first; tile < n_tiles && ok; tile += step) {
            const TcTile t = tc_tile<CG, BN>(p, tile);
            const int m = t.m0 + 128 * static_cast<int>(rank) + 32 * q + lane, n = t.n0 + half * S::HALF;
            const bool row = m < p.M;
            const float* sa = p.sa + static_cast<size_t>(row ? m : 0) * p.kb;
            const float* sb = p.sb + static_cast<size_t>(min(n, p.N - 1) / kQuantGroup) * p.kb;
            uint64_t acc[S::HALF / 2];
#pragma unroll
            for (int j = 0; j < S::HALF / 2; ++j) acc[j] = 0;
            float sa_next = __ldg(sa), sb_next = __ldg(sb);
            for (int b = 0; b < p.kb; ++b) {
                const float sc = sa_next * sb_next;
                if (b + 1 < p.kb) {
                    sa_next = __ldg(sa + b + 1);
                    sb_next = __ldg(sb + b + 1);
                }
                uint64_t s2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(sc));
                if (!mbar_wait(&s.tfull[buf], bphase, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < S::HALF; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(ta + buf * BN + c, r);
                    tmem_ld_wait_regs(r);
                    if (c + 32 == S::HALF) {  // the buffer is read: the next block's MMAs may have it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            // the reads are complete (tcgen05.wait::ld), so there is nothing to release
                            if (CG == 2) mbar_arrive_cluster_relaxed(tempty0 + buf * 8);
                            else mbar_arrive(&s.tempty[buf]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[c / 2 + j], s2, r[2 * j], r[2 * j + 1]);
                }
                if (++buf == S::NBUF) {
                    buf = 0;
                    bphase ^= 1;
                }
            }
            if (!ok) break;
            if (row) {
                const size_t at = static_cast<size_t>(m) * p.N + n;
#pragma unroll
                for (int c = 0; c < S::HALF; c += 8) {
                    if (n + c >= p.N) break;
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = __uint_as_float(static_cast<uint32_t>(acc[c / 2 + j]));
                        v[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(acc[c / 2 + j] >> 32));
                    }
                    if (p.addend) {
                        float f[8];
                        unpack8<ACT>(*reinterpret_cast<const uint4*>(p.addend + at + c), f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += f[j];
                    }
                    *reinterpret_cast<uint4*>(p.out + at + c) = pack8<ACT>(v);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();  // the leader's MMAs read this CTA's shared memory and write its TMEM
    tc_fence_after();
    if (warp == 1) {
        if (CG == 2) tmem_dealloc_pair(tmem, S::COLS);
        else tmem_dealloc(tmem, S::COLS);
    }
}

template <int ACT, int CG, int BN>
int launch_tc(const BfParams& p, int32_t* err, cudaStream_t st, const char* who) {
    using S = TcShape<CG, BN>;
    auto kernel = block_fp8_tc_kernel<ACT, CG, BN>;
    static int configured_for = -1;
    static int max_groups = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kTcThreads, 1, 1);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (configured_for != dev) {
        const int rc = set_smem_limit(reinterpret_cast<const void*>(kernel), S::SMEM);
        if (rc != MOE_OK) return rc;
        const int sms = sm_count();
        int n = sms;
        if (CG == 2) {
            cfg.gridDim = dim3(sms > 0 ? (sms / 2) * 2 : 2, 1, 1);
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess || n <= 0)
                return fail(MOE_ERR_CUDA, "%s: cannot place pairs of CTAs: %s", who, cudaGetErrorString(e));
        }
        max_groups = n;
        configured_for = dev;
    }
    CUtensorMap tm_a, tm_w;
    int rc = make_tmap_2d_u8(&tm_a, p.a, p.M, p.K, 128);
    if (rc == MOE_OK) rc = make_tmap_2d_u8(&tm_w, p.w, p.N, p.K, S::B_ROWS);
    if (rc != MOE_OK) return rc;
    const int64_t tiles = static_cast<int64_t>((p.M + 128 * CG - 1) / (128 * CG)) * ((p.N + BN - 1) / BN);
    if (tiles > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "%s: M=%d x N=%d is too large", who, p.M, p.N);
    cfg.gridDim = dim3(static_cast<unsigned>(CG * (tiles < max_groups ? tiles : max_groups)), 1, 1);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_w, p, err, wait_limit_ns());
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

template <int ACT> int pick_tc(const BfParams& p, int sms, int32_t* err, cudaStream_t st, const char* who) {
    // the pair's 256 x 256 tiles once they fill the GPU, else the narrower tiles that fill more of it
    const int64_t pairs = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + 255) / 256);
    if (2 * pairs >= sms) return launch_tc<ACT, 2, 256>(p, err, st, who);
    const int64_t mid = static_cast<int64_t>((p.M + 127) / 128) * ((p.N + 127) / 128);
    if (mid >= sms) return launch_tc<ACT, 1, 128>(p, err, st, who);
    return launch_tc<ACT, 1, 64>(p, err, st, who);
}

}  // namespace

int launch_block_fp8_tc(const BfParams& p, int act, int sms, int32_t* err, cudaStream_t st, const char* who) {
    return act == MOE_ACT_BF16 ? pick_tc<MOE_ACT_BF16>(p, sms, err, st, who)
                               : pick_tc<MOE_ACT_F16>(p, sms, err, st, who);
}

}  // namespace moe
