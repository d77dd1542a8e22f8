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
//   * Tokens sit on the products' 8-wide side: NT tiles of 8 rows of a; more
//     rows than 8 NT take further blocks (grid.y), which find the weights in L2.
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kBfThreads = 256, kBfWarps = kBfThreads / 32;
constexpr int kBfRing = 8;
constexpr int kBfSpan = 64;

struct BfParams {
    const uint8_t* a;
    const float* sa;
    const uint8_t* w;
    const float* sb;
    const uint16_t* addend;
    uint16_t* out;
    int M, N, K, kb;  // kb: scales per row
};

struct BfUnit {
    uint4 r[2];
    float s[2];
};

template <int ACT, int NT>
__global__ void __launch_bounds__(kBfThreads, 2) block_fp8_rows_kernel(const BfParams p) {
    __shared__ float4 red[kBfWarps * NT * 32];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
    const int m0 = blockIdx.y * 8 * NT;
    const int ms = min(8 * NT, p.M - m0);
    const int nt = (ms + 7) / 8;
    const int ntiles = (n1 - n0 + 15) / 16;
    const int K = p.K, nk = ((K + kBfSpan - 1) / kBfSpan + kBfWarps - 1) / kBfWarps;  // steps per warp and tile

    const uint8_t* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = 8 * t + g < ms ? p.a + static_cast<size_t>(m0 + 8 * t + g) * K : nullptr;

    BfUnit ring[kBfRing];
    int ltile = 0, lj = 0;
    auto fetch = [&](BfUnit& u) {
        if (ltile >= ntiles) return;
        const int k0 = (lj * kBfWarps + warp) * kBfSpan, k = k0 + 16 * c;
        const int ra = n0 + 16 * ltile + g, rb = ra + 8;
        u.r[0] = u.r[1] = make_uint4(0u, 0u, 0u, 0u);
        u.s[0] = u.s[1] = 0.0f;
        if (k < K && ra < n1) u.r[0] = ldg_stream16(p.w + static_cast<size_t>(ra) * K + k);
        if (k < K && rb < n1) u.r[1] = ldg_stream16(p.w + static_cast<size_t>(rb) * K + k);
        if (k0 < K && ra < n1) u.s[0] = __ldg(p.sb + static_cast<size_t>(ra / kQuantGroup) * p.kb + k0 / kQuantGroup);
        if (k0 < K && rb < n1) u.s[1] = __ldg(p.sb + static_cast<size_t>(rb / kQuantGroup) * p.kb + k0 / kQuantGroup);
        if (++lj == nk) {
            lj = 0;
            ++ltile;
        }
    };
#pragma unroll
    for (int d = 0; d < kBfRing; ++d) fetch(ring[d]);

    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
    int tile = 0, j = 0;
    while (tile < ntiles) {
#pragma unroll
        for (int d = 0; d < kBfRing; ++d) {
            if (tile >= ntiles) break;
            const int k0 = (j * kBfWarps + warp) * kBfSpan, k = k0 + 16 * c;
            if (k0 < K) {
                const BfUnit& u = ring[d];
                uint32_t fa[8], fb[8];
                const uint32_t wa[4] = {u.r[0].x, u.r[0].y, u.r[0].z, u.r[0].w};
                const uint32_t wb[4] = {u.r[1].x, u.r[1].y, u.r[1].z, u.r[1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e4m3x4_to_act<MOE_ACT_F16>(wa[i], fa[2 * i], fa[2 * i + 1]);
                    e4m3x4_to_act<MOE_ACT_F16>(wb[i], fb[2 * i], fb[2 * i + 1]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t >= nt) continue;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (xp[t] && k < K) x = __ldg(reinterpret_cast<const uint4*>(xp[t] + k));
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_act<MOE_ACT_F16>(xw[i], b0, b1);
                        mma_16816<MOE_ACT_F16>(part, fa[2 * i], fb[2 * i], fa[2 * i + 1], fb[2 * i + 1], b0, b1);
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int m = 8 * t + 2 * c + q;
                        const float sm =
                            m < ms ? __ldg(p.sa + static_cast<size_t>(m0 + m) * p.kb + k0 / kQuantGroup) : 0.0f;
                        acc[t][q] = fmaf(sm * u.s[0], part[q], acc[t][q]);
                        acc[t][2 + q] = fmaf(sm * u.s[1], part[2 + q], acc[t][2 + q]);
                    }
                }
            }
            if (++j == nk) {  // the tile's contraction is complete: add the warps' sums
                j = 0;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    red[(warp * NT + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                }
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
                        const size_t at = static_cast<size_t>(m0 + m) * p.N + n;
                        if (p.addend)
                            v += Act<ACT>::to_f(reinterpret_cast<const typename Act<ACT>::T*>(p.addend)[at]);
                        reinterpret_cast<typename Act<ACT>::T*>(p.out)[at] = Act<ACT>::from_f(v);
                    }
                }
                __syncthreads();
                ++tile;
            }
            fetch(ring[d]);
        }
    }
}

template <int ACT>
cudaError_t launch_rows(const BfParams& p, int sms, cudaStream_t st) {
    const int gx = sms < p.N ? sms : p.N;
    if (p.M <= 8) return launch_pdl(block_fp8_rows_kernel<ACT, 1>, dim3(gx), kBfThreads, 0, st, p);
    if (p.M <= 16) return launch_pdl(block_fp8_rows_kernel<ACT, 2>, dim3(gx), kBfThreads, 0, st, p);
    return launch_pdl(block_fp8_rows_kernel<ACT, 4>, dim3(gx, (p.M + 31) / 32), kBfThreads, 0, st, p);
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
    if (M > 65535 * 32) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: M=%d is too large", who, M);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(a && a_scales && w && w_scales && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(addend) && moe::aligned16(out),
                "%s: a / w / addend / out must be 16-byte aligned", who);
    MOE_REQUIRE(((reinterpret_cast<uintptr_t>(a_scales) | reinterpret_cast<uintptr_t>(w_scales)) & 3u) == 0,
                "%s: scales must be 4-byte aligned", who);
    (void)err_word;
    const int sms = moe::sm_count();
    if (sms <= 0) return moe::fail(MOE_ERR_CUDA, "%s: no CUDA device", who);
    const moe::BfParams p{static_cast<const uint8_t*>(a), a_scales, static_cast<const uint8_t*>(w), w_scales,
                          static_cast<const uint16_t*>(addend), static_cast<uint16_t*>(out), M, N, K,
                          (K + moe::kQuantGroup - 1) / moe::kQuantGroup};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = act == MOE_ACT_BF16 ? moe::launch_rows<MOE_ACT_BF16>(p, sms, st)
                                              : moe::launch_rows<MOE_ACT_F16>(p, sms, st);
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch();
    return moe::check_launch(who);
}
