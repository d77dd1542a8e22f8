// Rows form of the ragged products, fp16.
#include "ragged_tc.cuh"

int moe::launch_ragged_rows_f16(const RaggedArgs& g) {
    return g.transposed ? ragged::rows_form<MOE_ACT_F16, ragged::ROWS_BACK>(g)
                        : ragged::rows_form<MOE_ACT_F16, ragged::ROWS_FWD>(g);
}
