// Rows form of the ragged products, bf16 (a file for each type: they compile side by side).
#include "ragged_split.cuh"

int moe::launch_ragged_rows_bf16(const RaggedArgs& g, const RowsForm& f) {
    return ragged::launch_rows_act<MOE_ACT_BF16>(g, f);
}
