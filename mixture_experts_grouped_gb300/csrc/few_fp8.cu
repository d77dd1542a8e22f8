// The few-token layer on FP8 weights (few.cuh).
#include "few.cuh"

namespace moe {

cudaError_t launch_few_fp8(const FewParams& p, int act, int sms, cudaStream_t st) {
    return act == MOE_ACT_BF16 ? launch_few<MOE_W_FP8_E4M3, MOE_ACT_BF16>(p, sms, st)
                               : launch_few<MOE_W_FP8_E4M3, MOE_ACT_F16>(p, sms, st);
}

}  // namespace moe
