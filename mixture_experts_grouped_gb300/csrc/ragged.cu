// Products grouped by expert over ragged spans, their gradients, and the dense
// product with its epilogue: entry points.
#include "fn.cuh"

namespace moe {
namespace {

// D[i, j] = sum_k A(i, k) B(j, k), 64 x 64 a block, operands by strides. Plain f32
// multiply-adds from shared memory.
struct SimpleParams {
    const uint16_t *a, *b;
    const int32_t* offsets;
    int rows, E, I, J, K;                // I: -1 where i runs over a group's rows; K: -1 where k does
    int64_t ai, ak, ae, bj, bk, be;      // strides; per expert
    int64_t oi, oe;                      // output strides (j contiguous)
    void* out;
    const float* addend;
    const uint16_t *bias, *residual;
    uint16_t* pre;
    int fn, f32;
    int32_t* err;
};

template <int ACT>
__global__ void __launch_bounds__(256) simple_kernel(const SimpleParams p) {
    pdl_wait();
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    using T = typename Act<ACT>::T;
    if (p.offsets) {
        bool bad = p.offsets[0] < 0 || p.offsets[p.E] > p.rows;
        for (int e = 0; e < p.E; ++e) bad |= p.offsets[e + 1] < p.offsets[e];
        if (bad) {
            if (threadIdx.x == 0) set_err(p.err, MOE_DEV_ERR_OFFSETS);
            return;
        }
    }
    for (int e = blockIdx.z; e < p.E; e += gridDim.z) {
        const int r0 = p.offsets ? p.offsets[e] : 0, r1 = p.offsets ? p.offsets[e + 1] : p.rows;
        const int I = p.I < 0 ? r1 - r0 : p.I, K = p.K < 0 ? r1 - r0 : p.K;
        const int64_t abase = e * p.ae + (p.I < 0 ? r0 * p.ai : r0 * p.ak);
        const int64_t bbase = e * p.be + (p.K < 0 ? r0 * p.bk : 0);
        for (int i0 = blockIdx.y * 64; i0 < I; i0 += gridDim.y * 64) {
            const int j0 = blockIdx.x * 64;
            float acc[4][4] = {};
            for (int k0 = 0; k0 < K; k0 += 16) {
                for (int x = threadIdx.x; x < 1024; x += 256) {
                    const int kk = x & 15, i = x >> 4;
                    sa[kk][i] = i0 + i < I && k0 + kk < K
                                    ? Act<ACT>::to_f(reinterpret_cast<const T*>(p.a)[abase + (i0 + i) * p.ai + (k0 + kk) * p.ak])
                                    : 0.0f;
                    sb[kk][i] = j0 + i < p.J && k0 + kk < K
                                    ? Act<ACT>::to_f(reinterpret_cast<const T*>(p.b)[bbase + (j0 + i) * p.bj + (k0 + kk) * p.bk])
                                    : 0.0f;
                }
                __syncthreads();
                for (int kk = 0; kk < 16; ++kk)
                    for (int u = 0; u < 4; ++u)
                        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(sa[kk][ty * 4 + u], sb[kk][tx * 4 + v], acc[u][v]);
                __syncthreads();
            }
            for (int u = 0; u < 4; ++u)
                for (int v = 0; v < 4; ++v) {
                    const int i = i0 + ty * 4 + u, j = j0 + tx * 4 + v;
                    if (i >= I || j >= p.J) continue;
                    const int64_t at = e * p.oe + (p.I < 0 ? r0 + i : i) * p.oi + j;
                    float z = acc[u][v];
                    if (p.addend) z += p.addend[at];
                    if (p.bias) z += Act<ACT>::to_f(reinterpret_cast<const T*>(p.bias)[j]);
                    if (p.pre) reinterpret_cast<T*>(p.pre)[at] = Act<ACT>::from_f(z);
                    z = fn_value(p.fn, z);
                    if (p.residual) z += Act<ACT>::to_f(reinterpret_cast<const T*>(p.residual)[at]);
                    if (p.f32) static_cast<float*>(p.out)[at] = z;
                    else static_cast<T*>(p.out)[at] = Act<ACT>::from_f(z);
                }
        }
    }
}

int launch_simple(const SimpleParams& p, int act, int rows_i, void* stream, const char* who) {
    const dim3 grid((p.J + 63) / 64, rows_i < 64 * 1024 ? (rows_i + 63) / 64 : 1024, p.E);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = act == MOE_ACT_BF16 ? launch_pdl(simple_kernel<MOE_ACT_BF16>, grid, 256, 0, st, p)
                                              : launch_pdl(simple_kernel<MOE_ACT_F16>, grid, 256, 0, st, p);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

int check_shapes(const char* who, int act, const int32_t* offsets, int rows, int N, int K, int E) {
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(rows >= 0, "%s: %d rows", who, rows);
    MOE_REQUIRE(N > 0 && N % 8 == 0, "%s: N=%d must be a positive multiple of 8", who, N);
    MOE_REQUIRE(K > 0 && K % 8 == 0, "%s: K=%d must be a positive multiple of 8", who, K);
    MOE_REQUIRE(E >= 1 && E <= MOE_MAX_EXPERTS, "%s: E=%d outside [1, %d]", who, E, MOE_MAX_EXPERTS);
    MOE_REQUIRE(offsets || E == 1, "%s: no offsets, but E=%d groups", who, E);
    MOE_REQUIRE((reinterpret_cast<uintptr_t>(offsets) & 3u) == 0, "%s: offsets must be 4-byte aligned", who);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_ragged_gemm(const void* a, int32_t act, const void* w, int32_t transposed, const int32_t* offsets,
                               int32_t rows, int32_t N, int32_t K, int32_t E, void* out, int32_t* err_word,
                               void* stream) {
    const char* who = "moe_ragged_gemm";
    const int rc = moe::check_shapes(who, act, offsets, rows, N, K, E);
    if (rc != MOE_OK) return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(a && w && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(out), "%s: a / w / out must be 16-byte aligned",
                who);
    moe::SimpleParams p{};
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(w);
    p.offsets = offsets;
    p.rows = rows;
    p.E = E;
    p.I = -1;
    p.J = transposed ? K : N;
    p.K = transposed ? N : K;
    p.ai = p.K;
    p.ak = 1;
    p.bj = transposed ? 1 : K;
    p.bk = transposed ? K : 1;
    p.be = static_cast<int64_t>(N) * K;
    p.oi = p.J;
    p.out = out;
    p.err = err_word;
    return moe::launch_simple(p, act, rows, stream, who);
}

extern "C" int moe_ragged_wgrad(const void* dy, const void* x, int32_t act, const int32_t* offsets, int32_t rows,
                                int32_t N, int32_t K, int32_t E, const float* addend, void* dw, int32_t dw_f32,
                                int32_t* err_word, void* stream) {
    const char* who = "moe_ragged_wgrad";
    const int rc = moe::check_shapes(who, act, offsets, rows, N, K, E);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(dw_f32 || !addend, "%s: an addend goes with an f32 gradient", who);
    MOE_REQUIRE(dw && (rows == 0 || (dy && x)), "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(dy) && moe::aligned16(x) && moe::aligned16(addend) && moe::aligned16(dw),
                "%s: tensors must be 16-byte aligned", who);
    moe::SimpleParams p{};
    p.a = static_cast<const uint16_t*>(dy);
    p.b = static_cast<const uint16_t*>(x);
    p.offsets = offsets;
    p.rows = rows;
    p.E = E;
    p.I = N;
    p.J = K;
    p.K = -1;
    p.ai = 1;
    p.ak = N;
    p.bj = 1;
    p.bk = K;
    p.oi = K;
    p.oe = static_cast<int64_t>(N) * K;
    p.out = dw;
    p.addend = addend;
    p.f32 = dw_f32;
    p.err = err_word;
    return moe::launch_simple(p, act, N, stream, who);
}

extern "C" int moe_dense_gemm(const void* a, int32_t act, const void* w, const void* bias, int32_t fn,
                              const void* residual, void* pre, void* out, int32_t M, int32_t N, int32_t K,
                              int32_t* err_word, void* stream) {
    const char* who = "moe_dense_gemm";
    const int rc = moe::check_shapes(who, act, nullptr, M, N, K, 1);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(fn >= MOE_FN_NONE && fn <= MOE_FN_SILU, "%s: unknown activation function %d", who, fn);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(a && w && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(bias) && moe::aligned16(residual) &&
                    moe::aligned16(pre) && moe::aligned16(out),
                "%s: tensors must be 16-byte aligned", who);
    moe::SimpleParams p{};
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(w);
    p.rows = M;
    p.E = 1;
    p.I = -1;
    p.J = N;
    p.K = K;
    p.ai = K;
    p.ak = 1;
    p.bj = K;
    p.bk = 1;
    p.oi = N;
    p.out = out;
    p.bias = static_cast<const uint16_t*>(bias);
    p.residual = static_cast<const uint16_t*>(residual);
    p.pre = static_cast<uint16_t*>(pre);
    p.fn = fn;
    p.err = err_word;
    return moe::launch_simple(p, act, M, stream, who);
}
