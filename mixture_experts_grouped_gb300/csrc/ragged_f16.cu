// Rows form of the ragged products, f16 (a file for each type: they compile side by side).
#include "ragged_split.cuh"

int moe::launch_ragged_rows_f16(const RaggedArgs& g, const RowsForm& f) {
    return ragged::launch_rows_act<MOE_ACT_F16>(g, f);
}
