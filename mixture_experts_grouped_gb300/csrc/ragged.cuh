// What the tensor-core kernels of the ragged products take (ragged_tc.cuh), and
// their launchers.
#pragma once

#include "fn.cuh"

namespace moe {

// rows form: out[r, j] over the rows of each group; gradient form: dw_e[n, k]
struct RaggedParams {
    const int32_t* offsets;  // [E + 1], or NULL: one group of all rows
    int rows, E;
    int J, C;                // rows form: output columns, contraction; gradient form: n, k
    int maxu;                // rows form: most units of 16 rows a tile has; gradient form: k columns a tile has
    void* out;
    const uint16_t *bias, *residual;  // rows form
    uint16_t* pre;
    int fn;
    const float* addend;  // gradient form
    int32_t* err;
    uint64_t wait_ns;
};

struct RaggedArgs {
    RaggedParams p;
    const void *a, *w;  // rows form: rows, weights [E, .., ..]; gradient form: dy, x
    int act, transposed, f32;
    int N, K;           // the weight's shape
    cudaStream_t st;
    const char* who;
};

// How a product of rows runs: on CTA pairs, row tiles of up to maxu units of 16 rows; or, with
// parts > 0, one group split: row tiles, and CTAs that share a tile's contraction.
struct RowsForm {
    int maxu, tiles, parts;
};

int launch_ragged_rows_bf16(const RaggedArgs& g, const RowsForm& f);
int launch_ragged_rows_f16(const RaggedArgs& g, const RowsForm& f);
int launch_dense_rows(const RaggedArgs& g);  // up to 32 rows, one group, not transposed
int launch_ragged_wgrad(const RaggedArgs& g);

}  // namespace moe
