// Products grouped by expert over ragged spans, their gradients, and the dense
// product with its epilogue: entry points.
#include "ragged.cuh"

namespace moe {
namespace {

int launch_rows(const RaggedArgs& g) {
    return g.act == MOE_ACT_BF16 ? launch_ragged_rows_bf16(g) : launch_ragged_rows_f16(g);
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
    moe::RaggedArgs g{};
    g.p.offsets = offsets;
    g.p.rows = rows;
    g.p.E = E;
    g.p.J = transposed ? K : N;
    g.p.C = transposed ? N : K;
    g.p.out = out;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = a;
    g.w = w;
    g.act = act;
    g.transposed = transposed;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    return moe::launch_rows(g);
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
    moe::RaggedArgs g{};
    g.p.offsets = offsets;
    g.p.rows = rows;
    g.p.E = E;
    g.p.J = N;
    g.p.C = K;
    g.p.out = dw;
    g.p.addend = addend;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = dy;
    g.w = x;
    g.act = act;
    g.f32 = dw_f32;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    return moe::launch_ragged_wgrad(g);
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
    moe::RaggedArgs g{};
    g.p.rows = M;
    g.p.E = 1;
    g.p.J = N;
    g.p.C = K;
    g.p.out = out;
    g.p.bias = static_cast<const uint16_t*>(bias);
    g.p.residual = static_cast<const uint16_t*>(residual);
    g.p.pre = static_cast<uint16_t*>(pre);
    g.p.fn = fn;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = a;
    g.w = w;
    g.act = act;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    return moe::launch_rows(g);
}
