// The few-token layer's entry points: checks, then the kernels of few.cuh.
#include "common.cuh"
#include "few_params.cuh"

namespace moe {

cudaError_t launch_few_bf16(const FewParams& p, int act, int sms, cudaStream_t st);
cudaError_t launch_few_fp8(const FewParams& p, int act, int sms, cudaStream_t st);
cudaError_t launch_few_nvfp4(const FewParams& p, int act, int sms, cudaStream_t st);
cudaError_t launch_few_gptq(const FewParams& p, int act, int sms, cudaStream_t st);

namespace {

// The same rules as the grouped GEMMs' for a weight [E, N, K].
int check_weight(const MoeWeight* w, int act, int N, int K, const char* what, const char* who) {
    MOE_REQUIRE(w && w->w, "%s: %s weight is NULL", who, what);
    MOE_REQUIRE(aligned16(w->w), "%s: %s weight must be 16-byte aligned", who, what);
    switch (w->format) {
        case MOE_W_BF16:
            MOE_REQUIRE(act == MOE_ACT_BF16, "%s: bf16 weights need bf16 activations", who);
            return MOE_OK;
        case MOE_W_GPTQ_INT4:
            MOE_REQUIRE(w->scales && w->zeros, "%s: GPTQ needs scales and zeros", who);
            MOE_REQUIRE(w->group_size > 0 && w->group_size % 64 == 0 && K % w->group_size == 0,
                        "%s: GPTQ group_size=%d must be a multiple of 64 dividing K=%d", who, w->group_size, K);
            MOE_REQUIRE(N % 32 == 0, "%s: GPTQ needs N=%d to be a multiple of 32", who, N);
            MOE_REQUIRE(aligned16(w->scales) && aligned16(w->zeros), "%s: GPTQ scales / zeros must be 16-byte aligned",
                        who);
            return MOE_OK;
        case MOE_W_NVFP4:
            MOE_REQUIRE(w->scales && w->scale2, "%s: NVFP4 needs scales and scale2", who);
            MOE_REQUIRE(aligned16(w->scales), "%s: NVFP4 scales must be 16-byte aligned", who);
            MOE_REQUIRE(K % 32 == 0 && N % 16 == 0, "%s: NVFP4 needs K=%d %% 32 == 0 and N=%d %% 16 == 0", who, K, N);
            return MOE_OK;
        case MOE_W_FP8_E4M3:
            MOE_REQUIRE(w->scales, "%s: FP8 needs scales", who);
            MOE_REQUIRE(K % 16 == 0, "%s: FP8 needs K=%d %% 16 == 0", who, K);
            MOE_REQUIRE((reinterpret_cast<uintptr_t>(w->scales) & 3u) == 0, "%s: FP8 scales must be 4-byte aligned",
                        who);
            return MOE_OK;
        default:
            return fail(MOE_ERR_INVALID, "%s: unknown weight format %d", who, w->format);
    }
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_few_tokens_workspace_size(int32_t T, int32_t top_k, int32_t I) {
    if (T < 0 || top_k < 0 || I < 0) return 0;
    return (static_cast<size_t>(T) * top_k * I * 2 + 255) / 256 * 256;
}

extern "C" int moe_few_tokens(const void* x, int32_t act, const float* logits, int32_t* topk_ids, float* topk_weights,
                              const MoeWeight* w_gate_up, const MoeWeight* w_down, int32_t T, int32_t top_k, int32_t H,
                              int32_t I, int32_t E, int32_t renormalize, void* out, int32_t* err_word,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "moe_few_tokens";
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(E >= 1 && E <= MOE_MAX_EXPERTS, "%s: E=%d outside [1, %d]", who, E, MOE_MAX_EXPERTS);
    MOE_REQUIRE(top_k >= 1 && top_k <= E && top_k <= MOE_MAX_TOPK, "%s: top_k=%d outside [1, min(E=%d, %d)]", who,
                top_k, E, MOE_MAX_TOPK);
    MOE_REQUIRE(T >= 0, "%s: T=%d is negative", who, T);
    if (T > MOE_MAX_FEW_TOKENS)
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: T=%d above %d tokens", who, T, MOE_MAX_FEW_TOKENS);
    MOE_REQUIRE(H > 0 && H % 8 == 0, "%s: H=%d must be a positive multiple of 8", who, H);
    MOE_REQUIRE(I > 0 && I % 8 == 0, "%s: I=%d must be a positive multiple of 8", who, I);
    if (static_cast<int64_t>(2) * I * H >= (int64_t{1} << 30))
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: an expert of H=%d x I=%d is too large", who, H, I);
    // the kernels count rows (entry of the plan, i) in 32 bits: touched experts, and one more entry per 8 of their pairs
    const int64_t pairs = static_cast<int64_t>(T) * top_k;
    if (((pairs < E ? pairs : E) + pairs / 8) * I >= (int64_t{1} << 31))
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: T=%d x top_k=%d pairs may touch too many rows of I=%d", who, T, top_k,
                         I);
    int rc = moe::check_weight(w_gate_up, act, 2 * I, H, "gate/up", who);
    if (rc == MOE_OK) rc = moe::check_weight(w_down, act, H, I, "down", who);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(w_gate_up->format == w_down->format, "%s: gate/up and down weights of different formats (%d, %d)", who,
                w_gate_up->format, w_down->format);
    MOE_REQUIRE(w_gate_up->format != MOE_W_GPTQ_INT4 || I % 32 == 0, "%s: GPTQ needs I=%d to be a multiple of 32", who,
                I);
    MOE_REQUIRE(w_gate_up->format != MOE_W_NVFP4 || I % 16 == 0, "%s: NVFP4 needs I=%d to be a multiple of 16", who,
                I);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && topk_ids && topk_weights && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(x) && moe::aligned16(out), "%s: x / out must be 16-byte aligned", who);
    const size_t need = moe_few_tokens_workspace_size(T, top_k, I);
    MOE_REQUIRE(workspace && workspace_bytes >= need && moe::aligned16(workspace),
                "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", who, need, workspace_bytes);
    const int sms = moe::sm_count();
    if (sms <= 0) return moe::fail(MOE_ERR_CUDA, "%s: no CUDA device", who);
    const moe::FewParams p{static_cast<const uint16_t*>(x), logits, topk_ids, topk_weights, T, top_k, H, I, E,
                           renormalize ? 1 : 0, *w_gate_up, *w_down, static_cast<uint16_t*>(workspace),
                           static_cast<uint16_t*>(out), err_word};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (w_gate_up->format) {
        case MOE_W_BF16: e = moe::launch_few_bf16(p, act, sms, st); break;
        case MOE_W_FP8_E4M3: e = moe::launch_few_fp8(p, act, sms, st); break;
        case MOE_W_NVFP4: e = moe::launch_few_nvfp4(p, act, sms, st); break;
        default: e = moe::launch_few_gptq(p, act, sms, st); break;
    }
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch(2);
    return moe::check_launch(who);
}
