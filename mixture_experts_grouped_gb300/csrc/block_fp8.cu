// E4M3 matrix product with block scales.
//
//     out[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in b} a[m, k] w[n, k]  (+ addend[m, n])
//
// Few rows: bound by the weight bytes, so the weights stream straight into the
// fragments of warp-level tensor-core products (stream.cuh). E4M3 values are
// exact in f16 and their products exact in f32; the sums of each unit of 64
// contraction indices are scaled in f32 before they are added.
//   * Each CTA takes an equal share of the weight rows, in tiles of 16; the
//     contraction steps of a tile are dealt to its 8 warps in turn, and the
//     warps' sums are added through shared memory in warp order.
//   * Tokens sit on the products' 8-wide side: NT tiles of 8 rows of a.
// More rows run on the 5th-generation tensor cores (block_fp8_tc.cu).
#include "block_fp8.cuh"
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kBfThreads = 256, kBfWarps = kBfThreads / 32;
constexpr int kBfSpan = 64;   // contraction indices per unit
constexpr int kBfRing = 8;    // stages of a warp's ring
constexpr int kBfRowsMost = 32;  // rows up to which this form is used

// A stage: 1 KB of weights, NT tiles of tokens, the tokens' scales, two weight scales.
template <int NT> struct BfStage {
    static constexpr int X_AT = 1024, SA_AT = X_AT + 512 * NT, SB_AT = SA_AT + 32 * NT, BYTES = SB_AT + 16;
};

template <int ACT, int NT>
__global__ void __launch_bounds__(kBfThreads, 1) block_fp8_rows_kernel(const BfParams p) {
    using S = BfStage<NT>;
    extern __shared__ uint8_t bf_smem[];
    __shared__ float4 red[kBfWarps * NT * 32];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
    const int ms = p.M;  // <= 8 NT
    const int nt = (ms + 7) / 8;
    const int ntiles = (n1 - n0 + 15) / 16;
    const int K = p.K, nks = (K + kBfSpan - 1) / kBfSpan;
    uint8_t* ring = bf_smem + warp * kBfRing * S::BYTES;

    // the warp's units: tile by tile, steps warp, warp + 8, ... of each
    int ltile = warp < nks ? 0 : ntiles, lks = warp;
    auto fetch = [&](int stage) {
        if (ltile < ntiles) {
            uint8_t* st = ring + stage * S::BYTES;
            const int k0 = lks * kBfSpan, k = k0 + 16 * c, b = k0 / kQuantGroup;
            const bool in = k < K;
            const int kk = in ? k : 0;
            const int ra = n0 + 16 * ltile + g, rb = ra + 8;
            if (ra < n1) cp_async16_zfill(st + 16 * lane, p.w + static_cast<size_t>(ra) * K + kk, in);
            if (rb < n1) cp_async16_zfill(st + 512 + 16 * lane, p.w + static_cast<size_t>(rb) * K + kk, in);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (8 * t + g < ms)
                    cp_async16_l1(st + S::X_AT + 512 * t + 16 * lane,
                                  p.a + static_cast<size_t>(8 * t + g) * K + kk, in);
            if (lane < ms) cp_async4(st + S::SA_AT + 4 * lane, p.sa + static_cast<size_t>(lane) * p.kb + b);
            // 16 consecutive rows lie in at most two blocks of 128
            if (lane < 2) {
                const int n = min(n0 + 16 * ltile + 15 * lane, n1 - 1);
                cp_async4(st + S::SB_AT + 4 * lane, p.sb + static_cast<size_t>(n / kQuantGroup) * p.kb + b);
            }
            lks += kBfWarps;
            if (lks >= nks) {
                lks = warp;
                ++ltile;
            }
        }
        cp_async_commit();
    };
    for (int d = 0; d < kBfRing - 1; ++d) fetch(d);

    int stage = 0;
    for (int tile = 0; tile < ntiles; ++tile) {
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
        const int first_block = (n0 + 16 * tile) / kQuantGroup;
        const bool a2 = (n0 + 16 * tile + g) / kQuantGroup != first_block;      // row g lies in the second block
        const bool b2 = (n0 + 16 * tile + 8 + g) / kQuantGroup != first_block;  // row g + 8
        for (int ks = warp; ks < nks; ks += kBfWarps) {
            __syncwarp();  // every lane is done with the stage refilled now
            fetch(stage == 0 ? kBfRing - 1 : stage - 1);
            cp_async_wait_group<kBfRing - 1>();
            __syncwarp();  // scales were copied by other lanes
            const uint8_t* st = ring + stage * S::BYTES;
            const uint4 ua = *reinterpret_cast<const uint4*>(st + 16 * lane);
            const uint4 ub = *reinterpret_cast<const uint4*>(st + 512 + 16 * lane);
            const float* sb = reinterpret_cast<const float*>(st + S::SB_AT);
            const float s0 = sb[a2], s1 = sb[b2];
            uint32_t fa[8], fb[8];
            const uint32_t wa[4] = {ua.x, ua.y, ua.z, ua.w}, wb[4] = {ub.x, ub.y, ub.z, ub.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e4m3x4_to_act<MOE_ACT_F16>(wa[i], fa[2 * i], fa[2 * i + 1]);
                e4m3x4_to_act<MOE_ACT_F16>(wb[i], fb[2 * i], fb[2 * i + 1]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= nt) continue;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (8 * t + g < ms) x = *reinterpret_cast<const uint4*>(st + S::X_AT + 512 * t + 16 * lane);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x0, x1;
                    e4m3x4_to_act<MOE_ACT_F16>(xw[i], x0, x1);
                    mma_16816<MOE_ACT_F16>(part, fa[2 * i], fb[2 * i], fa[2 * i + 1], fb[2 * i + 1], x0, x1);
                }
                // sums of tokens past the batch are never read, so their stale scales do no harm
                const float2 sm = *reinterpret_cast<const float2*>(st + S::SA_AT + 32 * t + 8 * c);
                acc[t][0] = fmaf(sm.x * s0, part[0], acc[t][0]);
                acc[t][1] = fmaf(sm.y * s0, part[1], acc[t][1]);
                acc[t][2] = fmaf(sm.x * s1, part[2], acc[t][2]);
                acc[t][3] = fmaf(sm.y * s1, part[3], acc[t][3]);
            }
            if (++stage == kBfRing) stage = 0;
        }
        // the tile's contraction is complete: add the warps' sums
#pragma unroll
        for (int t = 0; t < NT; ++t)
            red[(warp * NT + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        __syncthreads();
        for (int i = tid; i < ms * 16; i += kBfThreads) {
            const int m = i >> 4, r = i & 15, n = n0 + 16 * tile + r;
            // row r, column m & 7 of token tile m / 8: lane 4 (r & 7) + (m & 7) / 2, element 2 (r / 8) + (m & 1)
            const float* src = reinterpret_cast<const float*>(red + (m >> 3) * 32 + 4 * (r & 7) + ((m & 7) >> 1)) +
                               2 * (r >> 3) + (m & 1);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kBfWarps; ++w) v += src[w * NT * 128];
            if (n < n1) {
                const size_t at = static_cast<size_t>(m) * p.N + n;
                if (p.addend) v += Act<ACT>::to_f(reinterpret_cast<const typename Act<ACT>::T*>(p.addend)[at]);
                reinterpret_cast<typename Act<ACT>::T*>(p.out)[at] = Act<ACT>::from_f(v);
            }
        }
        __syncthreads();
    }
}

template <int ACT, int NT>
cudaError_t launch_rows_nt(const BfParams& p, dim3 grid, cudaStream_t st) {
    constexpr int smem = kBfWarps * kBfRing * BfStage<NT>::BYTES;
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
    if (M > moe::kBfRowsMost) return moe::launch_block_fp8_tc(p, act, sms, err_word, st, who);
    const cudaError_t e = act == MOE_ACT_BF16 ? moe::launch_rows<MOE_ACT_BF16>(p, sms, st)
                                              : moe::launch_rows<MOE_ACT_F16>(p, sms, st);
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch();
    return moe::check_launch(who);
}
