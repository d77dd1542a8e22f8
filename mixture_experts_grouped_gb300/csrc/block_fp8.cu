// E4M3 matrix product with block scales.
//
//     out[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in b} a[m, k] w[n, k]  (+ addend[m, n])
//
// Few rows: bound by the weight bytes, so the weights stream straight into the
// fragments of warp-level tensor-core products (see stream.cuh for the ring
// and the free choice of k order). The products take the E4M3 codes as they
// are (m16n8k32, f32 accumulation: exact products, and a sum of 448^2 and 31
// terms of 2^-6 comes out exact), so nothing is converted; the f16 form of the
// same product costs eight times as much per contraction index here, and took
// 38 us at M = 17, N = 4096, K = 14336.
//   * Each CTA takes an equal share of the weight rows, 32 at a time; a unit
//     is 32 rows x one block of 128 contraction indices, whose sums are scaled
//     in f32 before they are added. The blocks are dealt to the CTA's 8 warps
//     in turn, and the warps' sums added through shared memory in warp order.
//   * Tokens sit on the products' 8-wide side: NT tiles of 8 rows of a, read
//     once per unit for all its 32 weight rows.
//   * A sum takes its token's scale first, then its rows' (block_fp8.cuh says
//     where their product would not do). Where a token's scale lies outside
//     [2^-63, 2^65) and its sums are not zeros, which is only noted on the way,
//     the warp takes its sums of the tile again with more care. (The note costs 0
//     to 5%, the most at M = 1 and 8, N = 28672; a vote and a branch in every unit
//     took 7%. Rows of zeros, whose scale is 2^-126, cost nothing.)
// Measured: M = 1, N = 2816, K = 2048 3.1 us (0.85 of it for the bytes at HBM's
// rate: a launch, one round trip to HBM and the sum of the warps make the rest);
// M = 8, N = 28672, K = 4096 27.1 us, 4.4 TB/s: every 32 rows the warps meet.
// More rows run on the 5th-generation tensor cores (block_fp8_tc.cu).
#include "block_fp8.cuh"
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kBfThreads = 256, kBfWarps = kBfThreads / 32;

// Which form: up to 8 rows this one; up to 16, and up to 32 (the most it takes),
// while the weights are small, and for more than 16 rows the contraction short
// too, since its reads of the tokens grow with both. Measured here / on tcgen05,
// us: 6.8 / 7.9 at M = 16, N = K = 4096, 12.7 / 10.4 at M = 16, N = 8192, K = 4096;
// 5.2 / 5.8 at M = 17, N = 2816, K = 2048, 8.0 / 5.9 at M = 17, N = 8192, K = 1408;
// 5.5 / 5.9 at M = 24, N = 4096, K = 2048, 7.8 / 6.3 at N = 2048, K = 4096; 5.2 / 5.8
// at M = 32, N = 2816, K = 1408, 6.3 / 5.9 at N = 4096, K = 2048. (M = 8, N = 28672,
// K = 4096 would take 25.6 there, 27.1 here, and M = 4 25.6 and 23.9.)
inline bool rows_form(int M, int N, int K) {
    const int64_t weights = static_cast<int64_t>(N) * K;
    if (M <= 16) return M <= 8 || weights <= (1 << 24);
    return M <= 32 && weights <= (1 << 23) && static_cast<int64_t>(M) * K <= 49152;
}

// A stage: 4 KB of weights (32 rows x 128), NT tiles of 8 tokens, the tokens'
// scales, two weight scales. The ring has what fits 200 KB, at most 6 stages.
template <int NT> struct BfStage {
    static constexpr int X_AT = 4096, SA_AT = X_AT + 1024 * NT, SB_AT = SA_AT + 32 * NT, BYTES = SB_AT + 16;
    static constexpr int FIT = 204800 / (kBfWarps * BYTES), RING = FIT < 6 ? FIT : 6;
    // Sums of the warps. One token tile: of all 32 rows, in two areas in turn, one
    // barrier a tile (M = 1, N = 2816, K = 2048 3.1 us, 3.4 by 16 rows); with more
    // tokens 16 rows, two barriers (M = 16, N = K = 2048 3.8 us, 4.0 by 32).
    static constexpr int HALVES = NT == 1 ? 2 : 1, RED = kBfWarps * 512 * NT * HALVES * HALVES;
    static constexpr int SMEM = kBfWarps * RING * BYTES + RED;
    static_assert(SMEM <= 232448, "shared memory over the limit");
};

__device__ __forceinline__ void mma_e4m3_16832(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 0 where 2^-63 <= |s| < 2^65 (the exponent's two upper bits differ), else all ones
__device__ __forceinline__ uint32_t odd_mask(float s) {
    const uint32_t u = __float_as_uint(s);
    return ~static_cast<uint32_t>(static_cast<int32_t>((u ^ u << 1) << 1) >> 31);
}

// Sums of one block of 128: 32 weight rows (two halves of 16) x 8 tokens
__device__ __forceinline__ void block_sums(const uint4 (&w)[4][2], const uint4 (&x)[2], float (&part)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        part[h][0] = part[h][1] = part[h][2] = part[h][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mma_e4m3_16832(part[h], w[2 * h][i].x, w[2 * h + 1][i].x, w[2 * h][i].y, w[2 * h + 1][i].y, x[i].x, x[i].y);
            mma_e4m3_16832(part[h], w[2 * h][i].z, w[2 * h + 1][i].z, w[2 * h][i].w, w[2 * h + 1][i].w, x[i].z, x[i].w);
        }
    }
}

// One warp's sums of the tile of rows [first, n1), first + 32 at most, again and
// straight from global memory: for the scales that the kernel's own order of
// products does not suit (see there), with the care of scale_before.
template <int NT>
__device__ __noinline__ void careful_sums(const BfParams& p, int first, int n1, int warp, int lane,
                                          float (&acc)[2][NT][4]) {
    const int g = lane >> 2, c = lane & 3, ms = p.M;
    auto piece = [&](const uint8_t* rows, int row, int end, int k) {
        return row < end && k < p.K ? *reinterpret_cast<const uint4*>(rows + static_cast<size_t>(row) * p.K + k)
                                    : make_uint4(0u, 0u, 0u, 0u);
    };
    for (int h = 0; h < 2; ++h)
        for (int t = 0; t < NT; ++t) acc[h][t][0] = acc[h][t][1] = acc[h][t][2] = acc[h][t][3] = 0.0f;
    for (int b = warp; b < p.kb; b += kBfWarps) {
        const int k = b * kQuantGroup + 16 * c;
        uint4 w[4][2];
        float s[4];
        for (int r = 0; r < 4; ++r) {
            const int row = first + 8 * r + g;
            for (int i = 0; i < 2; ++i) w[r][i] = piece(p.w, row, n1, k + 64 * i);
            s[r] = p.sb[static_cast<size_t>(min(row, n1 - 1) / kQuantGroup) * p.kb + b];
        }
        for (int t = 0; t < NT && 8 * t < ms; ++t) {
            const uint4 x[2] = {piece(p.a, 8 * t + g, ms, k), piece(p.a, 8 * t + g, ms, k + 64)};
            float part[2][4];
            block_sums(w, x, part);
            for (int q = 0; q < 2; ++q) {
                const float sm = p.sa[static_cast<size_t>(min(8 * t + 2 * c + q, ms - 1)) * p.kb + b];
                for (int h = 0; h < 2; ++h)
                    for (int r = 0; r < 2; ++r) {
                        float f = sm * s[2 * h + r];
                        const float v = part[h][2 * r + q] * scale_before(f, sm, s[2 * h + r]);
                        acc[h][t][2 * r + q] = fmaf(v, f, acc[h][t][2 * r + q]);
                    }
            }
        }
    }
}

template <int ACT, int NT>
__global__ void __launch_bounds__(kBfThreads, 1) block_fp8_rows_kernel(const BfParams p) {
    using S = BfStage<NT>;
    constexpr int RING = S::RING;
    extern __shared__ uint8_t bf_smem[];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
    const int ms = p.M;  // <= 8 NT
    const int nt = (ms + 7) / 8;
    const int ntiles = (n1 - n0 + 31) / 32;
    const int K = p.K;
    uint8_t* ring = bf_smem + warp * RING * S::BYTES;
    float4* red = reinterpret_cast<float4*>(bf_smem + kBfWarps * RING * S::BYTES);  // [areas][halves][warps][NT][32]

    // Lane (g, c) copies and uses, of rows g, g + 8, g + 16, g + 24 and of token
    // g of each tile, the 16-byte pieces c and c + 4 of a block's 128 codes.
    const int row8 = 8 * K;  // bytes from a row to the one 8 below
    const uint8_t* const pa = p.a + static_cast<size_t>(g) * K + 16 * c;
    const float* const psa = p.sa + static_cast<size_t>(lane < ms ? lane : 0) * p.kb;
    const int tiles_mine = (ms - g + 7) / 8;  // token tiles in which this lane has a token (may be 0)
    const uint8_t* pw = nullptr;              // row g of the current tile
    const float* psb = nullptr;               // lanes 0 and 1: the tile's first and last block scales
    int rows_mine = 0;                        // of the lane's four rows
    auto aim = [&](int first) {
        pw = p.w + static_cast<size_t>(first + g) * K + 16 * c;
        rows_mine = (n1 - first - g + 7) / 8;
        // 32 consecutive rows lie in at most two blocks of 128
        psb = p.sb + static_cast<size_t>(min(first + 31 * (lane & 1), n1 - 1) / kQuantGroup) * p.kb;
    };
    auto fetch = [&](int stage, int b) {
        uint8_t* st = ring + stage * S::BYTES;
        const int k0 = b * kQuantGroup;
        if (k0 + kQuantGroup <= K) {
            uint8_t* d = st + 16 * lane;
            const uint8_t* w = pw + k0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (r < rows_mine) {
                    cp_async16(d + 1024 * r, w);
                    cp_async16(d + 1024 * r + 512, w + 64);
                }
                w += row8;
            }
            const uint8_t* a = pa + k0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t < tiles_mine) {
                    cp_async16_l1(d + S::X_AT + 1024 * t, a, true);
                    cp_async16_l1(d + S::X_AT + 1024 * t + 512, a + 64, true);
                }
                a += row8;
            }
        } else {  // the last block of a K that 128 does not divide: zeros past its end
            const bool in0 = k0 + 16 * c < K, in1 = k0 + 64 + 16 * c < K;
            const int o0 = in0 ? k0 : 0, o1 = in1 ? k0 + 64 : 0;
            for (int r = 0; r < min(4, rows_mine); ++r) {
                cp_async16_zfill(st + 1024 * r + 16 * lane, pw + static_cast<size_t>(r) * row8 + o0, in0);
                cp_async16_zfill(st + 1024 * r + 512 + 16 * lane, pw + static_cast<size_t>(r) * row8 + o1, in1);
            }
            for (int t = 0; t < min(NT, tiles_mine); ++t) {
                cp_async16_l1(st + S::X_AT + 1024 * t + 16 * lane, pa + static_cast<size_t>(t) * row8 + o0, in0);
                cp_async16_l1(st + S::X_AT + 1024 * t + 512 + 16 * lane, pa + static_cast<size_t>(t) * row8 + o1, in1);
            }
        }
        if (lane < ms) cp_async4(st + S::SA_AT + 4 * lane, psa + b);
        if (lane < 2) cp_async4(st + S::SB_AT + 4 * lane, psb + b);
    };

    // the warp's units: blocks warp, warp + 8, ... of each tile; the copies run on into the next tile
    int ltile = warp < p.kb ? 0 : ntiles, lb = warp;
    if (ltile < ntiles) aim(n0);
    auto copy_next = [&](int stage) {
        if (ltile < ntiles) {
            fetch(stage, lb);
            lb += kBfWarps;
            if (lb >= p.kb) {
                lb = warp;
                if (++ltile < ntiles) aim(n0 + 32 * ltile);
            }
        }
        cp_async_commit();
    };
    // no copy brings scales of tokens past the batch; their sums are never read, but must not look odd below
    if (lane >= ms && lane < 8 * NT)
        for (int d = 0; d < RING; ++d) *reinterpret_cast<float*>(ring + d * S::BYTES + S::SA_AT + 4 * lane) = 1.0f;
    for (int d = 0; d < RING - 1; ++d) copy_next(d);
    int stage = 0;
    for (int tile = 0; tile < ntiles; ++tile) {
        const int first = n0 + 32 * tile;
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[h][t][0] = acc[h][t][1] = acc[h][t][2] = acc[h][t][3] = 0.0f;
        // of the lane's rows, not 0: a token's scale is out of the ordinary where its sum is not 0
        uint32_t odd[4] = {0u, 0u, 0u, 0u};
        // which of the two weight scales each of the lane's rows takes
        const int border = (first / kQuantGroup + 1) * kQuantGroup - first;  // rows before the second block
        for (int b = warp; b < p.kb; b += kBfWarps) {
            __syncwarp();  // every lane is done with the stage refilled now
            copy_next(stage == 0 ? RING - 1 : stage - 1);
            cp_async_wait_group<RING - 1>();
            __syncwarp();  // scales were copied by other lanes
            const uint8_t* st = ring + stage * S::BYTES;
            if (++stage == RING) stage = 0;
            uint4 w[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[r][i] = *reinterpret_cast<const uint4*>(st + 1024 * r + 512 * i + 16 * lane);
            const float2 sb = *reinterpret_cast<const float2*>(st + S::SB_AT);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= nt) break;
                uint4 x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    x[i] = 8 * t + g < ms ? *reinterpret_cast<const uint4*>(st + S::X_AT + 1024 * t + 512 * i + 16 * lane)
                                          : make_uint4(0u, 0u, 0u, 0u);
                const float2 sm = *reinterpret_cast<const float2*>(st + S::SA_AT + 32 * t + 8 * c);
                float part[2][4];
                block_sums(w, x, part);
                // (sum * token's scale) * rows' scale: each product is exact enough, whatever the rows' scale,
                // while the token's keeps the first one in the normal range
                const uint32_t mx = odd_mask(sm.x), my = odd_mask(sm.y);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    odd[r] |= __float_as_uint(part[r >> 1][2 * (r & 1)]) & mx;
                    odd[r] |= __float_as_uint(part[r >> 1][2 * (r & 1) + 1]) & my;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float s0 = 16 * h + g < border ? sb.x : sb.y, s1 = 16 * h + 8 + g < border ? sb.x : sb.y;
                    acc[h][t][0] = fmaf(part[h][0] * sm.x, s0, acc[h][t][0]);
                    acc[h][t][1] = fmaf(part[h][1] * sm.y, s0, acc[h][t][1]);
                    acc[h][t][2] = fmaf(part[h][2] * sm.x, s1, acc[h][t][2]);
                    acc[h][t][3] = fmaf(part[h][3] * sm.y, s1, acc[h][t][3]);
                }
            }
        }
        const int left = n1 - first - g;  // (rows past the share hold whatever their stage held)
        if (__any_sync(0xffffffffu, (left > 0 && odd[0]) || (left > 8 && odd[1]) || (left > 16 && odd[2]) ||
                                        (left > 24 && odd[3]))) {
            float again[2][NT][4];  // (acc itself stays in registers)
            careful_sums<NT>(p, first, n1, warp, lane, again);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[h][t][q] = again[h][t][q];
        }
        // the tile's contraction is complete: add the warps' sums, HALVES x 16 rows at a time
        constexpr int HALVES = S::HALVES;
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += HALVES) {
            if (first + 16 * h0 >= n1) break;
            float4* area = red + (HALVES == 2 ? tile & 1 : 0) * HALVES * kBfWarps * NT * 32;
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < nt)
                        area[((h * kBfWarps + warp) * NT + t) * 32 + lane] = make_float4(
                            acc[h0 + h][t][0], acc[h0 + h][t][1], acc[h0 + h][t][2], acc[h0 + h][t][3]);
            __syncthreads();
            for (int i = tid; i < ms * 16 * HALVES; i += kBfThreads) {
                const int r = i % (16 * HALVES), m = i / (16 * HALVES), h = r >> 4, n = first + 16 * h0 + r;
                // row r & 15, column m & 7 of token tile m / 8: lane 4 (r & 7) + (m & 7) / 2, element 2 (r / 8 & 1) + (m & 1)
                const float* src =
                    reinterpret_cast<const float*>(area + (h * kBfWarps * NT + (m >> 3)) * 32 + 4 * (r & 7) +
                                                   ((m & 7) >> 1)) +
                    2 * ((r >> 3) & 1) + (m & 1);
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kBfWarps; ++w) v += src[w * NT * 128];
                if (n < n1) {
                    const size_t at = static_cast<size_t>(m) * p.N + n;
                    if (p.addend) v += Act<ACT>::to_f(reinterpret_cast<const typename Act<ACT>::T*>(p.addend)[at]);
                    reinterpret_cast<typename Act<ACT>::T*>(p.out)[at] = Act<ACT>::from_f(v);
                }
            }
            if (HALVES == 1) __syncthreads();  // with two areas the next tile's barrier parts a reader and the next writer
        }
    }
}

template <int ACT, int NT>
cudaError_t launch_rows_nt(const BfParams& p, dim3 grid, cudaStream_t st) {
    constexpr int smem = BfStage<NT>::SMEM;
    static int configured_for = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        if (set_smem_limit(reinterpret_cast<const void*>(block_fp8_rows_kernel<ACT, NT>), smem) != MOE_OK)
            return cudaGetLastError();
        configured_for = dev;
    }
    return launch_pdl(block_fp8_rows_kernel<ACT, NT>, grid, kBfThreads, smem, st, p);
}

template <int ACT>
cudaError_t launch_rows(const BfParams& p, int sms, cudaStream_t st) {
    const int gx = sms < p.N ? sms : p.N;
    if (p.M <= 8) return launch_rows_nt<ACT, 1>(p, dim3(gx), st);
    if (p.M <= 16) return launch_rows_nt<ACT, 2>(p, dim3(gx), st);
    return launch_rows_nt<ACT, 4>(p, dim3(gx), st);
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_fp8_gemm(const void* a, const float* a_scales, const void* w, const float* w_scales,
                                  const void* addend, void* out, int32_t act, int32_t M, int32_t N, int32_t K,
                                  int32_t* err_word, void* stream) {
    const char* who = "moe_block_fp8_gemm";
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(M >= 0, "%s: M=%d is negative", who, M);
    MOE_REQUIRE(N > 0 && N % 8 == 0, "%s: N=%d must be a positive multiple of 8", who, N);
    MOE_REQUIRE(K > 0 && K % 16 == 0, "%s: K=%d must be a positive multiple of 16", who, K);
    if (M > (1 << 30) || N > (1 << 30) || K > (1 << 27))
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: M=%d, N=%d or K=%d is too large", who, M, N, K);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(a && a_scales && w && w_scales && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(addend) && moe::aligned16(out),
                "%s: a / w / addend / out must be 16-byte aligned", who);
    MOE_REQUIRE(((reinterpret_cast<uintptr_t>(a_scales) | reinterpret_cast<uintptr_t>(w_scales)) & 3u) == 0,
                "%s: scales must be 4-byte aligned", who);
    const int sms = moe::sm_count();
    if (sms <= 0) return moe::fail(MOE_ERR_CUDA, "%s: no CUDA device", who);
    const moe::BfParams p{static_cast<const uint8_t*>(a), a_scales, static_cast<const uint8_t*>(w), w_scales,
                          static_cast<const uint16_t*>(addend), static_cast<uint16_t*>(out), M, N, K,
                          (K + moe::kQuantGroup - 1) / moe::kQuantGroup};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!moe::rows_form(M, N, K)) return moe::launch_block_fp8_tc(p, act, sms, err_word, st, who);
    const cudaError_t e = act == MOE_ACT_BF16 ? moe::launch_rows<MOE_ACT_BF16>(p, sms, st)
                                              : moe::launch_rows<MOE_ACT_F16>(p, sms, st);
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch();
    return moe::check_launch(who);
}
