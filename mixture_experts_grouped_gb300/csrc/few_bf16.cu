// The few-token layer on bf16 weights (few.cuh).
#include "few.cuh"

namespace moe {

cudaError_t launch_few_bf16(const FewParams& p, int act, int sms, cudaStream_t st) {
    (void)act;  // bf16 weights come with bf16 activations
    return launch_few<MOE_W_BF16, MOE_ACT_BF16>(p, sms, st);
}

}  // namespace moe
