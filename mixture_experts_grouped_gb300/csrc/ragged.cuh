// What the tensor-core kernels of the ragged products take (ragged_tc.cuh), and
// their launchers.
#pragma once

#include "fn.cuh"

namespace moe {

// x / d of 0 <= x < 2^31 by a multiplication (m = floor(2^(31 + s) / d) + 1, 2^s >= d: the quotient's error
// stays below x / 2^31 steps of 1 / d)
struct FastDiv {
    uint32_t m, s, d;
    void set(uint32_t div) {
        d = div;
        s = 0;
        while ((1ull << s) < div) ++s;
        m = static_cast<uint32_t>((1ull << (31 + s)) / div + 1);
    }
    __device__ __forceinline__ int div(int x) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * m) >> (31 + s));
    }
};

// rows form: out[r, j] over the rows of each group; gradient form: dw_e[n, k]
struct RaggedParams {
    const int32_t* offsets;  // [E + 1], or NULL: one group of all rows
    int rows, E;
    int J, C;                // rows form: output columns, contraction; gradient form: n, k
    int maxu;                // rows form: most units of 16 rows a tile has
    FastDiv units;           // rows form: by maxu
    FastDiv kt, per;         // gradient form: tiles of a row of tiles, and of a group
    int kunit, kleast, kmore;  // a row's tiles are kleast units of kunit columns wide, the first kmore one more
    int turn;                // places by which a pair's tile moves on in each wave of tiles
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
    int parts;          // gradient form: CTAs that share a tile's contraction; 0: CTA pairs,
    int kt;             // with this many tiles side by side
    cudaStream_t st;
    const char* who;
};

// Columns that the width of a gradient's tile is a multiple of: a store's 128 bytes.
constexpr int gradient_unit(bool f32) { return f32 ? 32 : 64; }

// Most blocks of 64 rows that one accumulator of a gradient sums, since a tensor core's sums
// of n rows may come out n 2^-27 short (ragged_tc.cuh). For f32 640 rows: of random signs they
// are off by 8e-7 of their 2-norm in f16 and 6e-7 in bf16, as good as a plain f32 product; 4096
// rows by 5e-6. For 16 bits as many as lose a quarter of the output's half step (2^-13 of 2^-11
// in f16, 2^-10 of 2^-8 in bf16); without that, 1.2 million rows of one sign came out 0.8% short.
constexpr int gradient_chunk(bool f32, int act) { return f32 ? 10 : act == MOE_ACT_F16 ? 256 : 2048; }

// How a product of rows runs: on CTA pairs, row tiles of up to maxu units of 16 rows; or, with
// parts > 0, split: row tiles, and CTAs that share a tile's contraction.
struct RowsForm {
    int maxu, tiles, parts;
};
constexpr int SPLIT_MAX_ROWS = 128;  // most rows of groups that the split form takes

// What a kernel's first launch on a device found out or set (0: not yet), for launches from any thread.
struct PerDevice {
    std::atomic<int> of[64] = {};
    std::atomic<int>* here() {
        int dev = 0;
        return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? &of[dev] : nullptr;
    }
};
// the kernel's limit of dynamic shared memory, raised once a device
inline int raise_smem_limit(PerDevice& done, const void* kernel, int bytes) {
    std::atomic<int>* d = done.here();
    if (d && d->load(std::memory_order_acquire)) return MOE_OK;
    const int rc = set_smem_limit(kernel, bytes);
    if (rc == MOE_OK && d) d->store(1, std::memory_order_release);
    return rc;
}

int launch_ragged_rows_bf16(const RaggedArgs& g, const RowsForm& f);
int launch_ragged_rows_f16(const RaggedArgs& g, const RowsForm& f);
int launch_dense_rows(const RaggedArgs& g);  // up to 32 rows, one group, not transposed
int launch_ragged_wgrad(const RaggedArgs& g);

}  // namespace moe
