// Rows form of the ragged products, bf16.
#include "ragged_split.cuh"

int moe::launch_ragged_rows_bf16(const RaggedArgs& g, const RowsForm& f) {
    constexpr int ACT = MOE_ACT_BF16;
    if (f.parts) {
        return g.transposed ? ragged::launch_split<ragged::ROWS_BACK, ACT>(g, f.tiles, f.parts)
                            : ragged::launch_split<ragged::ROWS_FWD, ACT>(g, f.tiles, f.parts);
    }
    return g.transposed ? ragged::launch_rows_form<ragged::ROWS_BACK, ACT>(g, f.maxu)
                        : ragged::launch_rows_form<ragged::ROWS_FWD, ACT>(g, f.maxu);
}
