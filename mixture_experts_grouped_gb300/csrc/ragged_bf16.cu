// Rows form of the ragged products, bf16.
#include "ragged_tc.cuh"

int moe::launch_ragged_rows_bf16(const RaggedArgs& g) {
    return g.transposed ? ragged::rows_form<MOE_ACT_BF16, ragged::ROWS_BACK>(g)
                        : ragged::rows_form<MOE_ACT_BF16, ragged::ROWS_FWD>(g);
}
