// Dense product of few rows with its epilogue (see moe_dense_gemm), streaming form.
//
//     z[m, n] = sum_k a[m, k] w[n, k] + bias[n],   out = f(z) + residual
//
// Bound by the weights' bytes and, where they are few, by latency: weights stream by
// cp.async into rings private to a warp and go as they are into the fragments of
// warp-level products (m16n8k16; the order of the contraction is free, see stream.cuh),
// without barriers, tensor maps or tensor memory to set up. Each CTA takes an equal share
// of the weight rows, 32 at a time; a unit is 32 rows x 64 contraction indices; the blocks of
// 64 are dealt to the CTA's 8 warps in turn, and the warps' sums added through shared
// memory in warp order. Tokens sit on the products' 8-wide side, NT tiles of 8.
// Measured: 1 x 2816 x 2048 4.8 us, 3 x 2048 x 1408 4.0 (1.7 and 0.9 for the bytes: a
// launch, a round trip to HBM and the warps' sum make the rest); 1 x 4096 x 14336 22.4 us, 5.2
// TB/s; 16 rows 26, 32 rows 38, where the rows that every CTA reads from L2 bound it, and the
// split form (ragged_split.cuh) takes 26. ragged.cu has the choice.
#include "ragged.cuh"
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct DenseRowsParams {
    const uint16_t *a, *w;
    int M, N, K, kb;
    RaggedParams r;
};

template <int NT> struct RowsStage {
    static constexpr int X_AT = 4096, BYTES = X_AT + 1024 * NT;
    static constexpr int FIT = 196608 / (kWarps * BYTES), RING = FIT < 6 ? FIT : 6;
    static constexpr int RED = kWarps * 32 * 8 * NT * 4;  // the warps' sums of a tile
    static constexpr int SMEM = kWarps * RING * BYTES + RED;
    static_assert(RING >= 3 && SMEM <= 232448, "shared memory over the limit");
};

template <int ACT, int NT>
__global__ void __launch_bounds__(kThreads, 1) dense_rows_kernel(const DenseRowsParams p) {
    using S = RowsStage<NT>;
    using T = typename Act<ACT>::T;
    constexpr int RING = S::RING;
    extern __shared__ uint8_t dr_smem[];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
    const int n1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
    const int M = p.M, nt = (M + 7) / 8, ntiles = (n1 - n0 + 31) / 32;
    const size_t K = p.K, row8 = 8 * K;
    uint8_t* ring = dr_smem + warp * RING * S::BYTES;
    float* red = reinterpret_cast<float*>(dr_smem + kWarps * RING * S::BYTES);  // [warps][2][NT][32][4]

    // Lane (g, c) copies and uses, of rows g, g + 8, g + 16, g + 24 and of token g of each
    // tile, the 16-byte pieces c and c + 4 of a block's 128 bytes.
    const uint16_t* const pa = p.a + static_cast<size_t>(g) * K + 8 * c;
    const int tiles_mine = (M - g + 7) / 8;  // token tiles in which this lane has a token
    const uint16_t* pw = nullptr;
    int rows_mine = 0;
    auto aim = [&](int first) {
        pw = p.w + static_cast<size_t>(first + g) * K + 8 * c;
        rows_mine = (n1 - first - g + 7) / 8;
    };
    auto fetch = [&](int stage, int b) {
        uint8_t* d = ring + stage * S::BYTES + 16 * lane;
        const int k0 = b * 64;
        if (k0 + 64 <= p.K) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < rows_mine) {
                    cp_async16_row(d + 1024 * r, pw + r * row8 + k0);
                    cp_async16_row(d + 1024 * r + 512, pw + r * row8 + k0 + 32);
                }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < tiles_mine) {
                    cp_async16_l1(d + S::X_AT + 1024 * t, pa + t * row8 + k0, true);
                    cp_async16_l1(d + S::X_AT + 1024 * t + 512, pa + t * row8 + k0 + 32, true);
                }
        } else {  // the last block of a K that 64 does not divide: zeros past its end
            const bool in0 = k0 + 8 * c < p.K, in1 = k0 + 32 + 8 * c < p.K;
            const int o0 = in0 ? k0 : 0, o1 = in1 ? k0 + 32 : 0;
            for (int r = 0; r < min(4, rows_mine); ++r) {
                cp_async16_zfill(d + 1024 * r, pw + r * row8 + o0, in0);
                cp_async16_zfill(d + 1024 * r + 512, pw + r * row8 + o1, in1);
            }
            for (int t = 0; t < min(NT, tiles_mine); ++t) {
                cp_async16_l1(d + S::X_AT + 1024 * t, pa + t * row8 + o0, in0);
                cp_async16_l1(d + S::X_AT + 1024 * t + 512, pa + t * row8 + o1, in1);
            }
        }
    };
    // the warp's units: blocks warp, warp + 8, ... of each tile; the copies run on into the next tile
    int ltile = warp < p.kb ? 0 : ntiles, lb = warp;
    if (ltile < ntiles) aim(n0);
    auto copy_next = [&](int stage) {
        if (ltile < ntiles) {
            fetch(stage, lb);
            lb += kWarps;
            if (lb >= p.kb) {
                lb = warp;
                if (++ltile < ntiles) aim(n0 + 32 * ltile);
            }
        }
        cp_async_commit();
    };
    for (int d = 0; d < RING - 1; ++d) copy_next(d);
    int stage = 0;
    for (int tile = 0; tile < ntiles; ++tile) {
        const int first = n0 + 32 * tile;
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[h][t][0] = acc[h][t][1] = acc[h][t][2] = acc[h][t][3] = 0.0f;
        for (int b = warp; b < p.kb; b += kWarps) {
            copy_next(stage == 0 ? RING - 1 : stage - 1);  // (a lane reads only what it copied itself)
            cp_async_wait_group<RING - 1>();
            const uint8_t* st = ring + stage * S::BYTES + 16 * lane;
            if (++stage == RING) stage = 0;
            // (rows and tokens that there are not give whatever the stage held to sums that nobody reads)
            uint4 w[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[r][i] = *reinterpret_cast<const uint4*>(st + 1024 * r + 512 * i);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= nt) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4*>(st + S::X_AT + 1024 * t + 512 * i);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma_16816<ACT>(acc[h][t], w[2 * h][i].x, w[2 * h + 1][i].x, w[2 * h][i].y, w[2 * h + 1][i].y, x.x,
                                       x.y);
                        mma_16816<ACT>(acc[h][t], w[2 * h][i].z, w[2 * h + 1][i].z, w[2 * h][i].w, w[2 * h + 1][i].w, x.z,
                                       x.w);
                    }
                }
            }
        }
        // the tile's contraction is complete: add the warps' sums
        if (tile > 0) __syncthreads();  // the last tile's are read
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t < nt)
                    *reinterpret_cast<float4*>(red + (((warp * 2 + h) * NT + t) * 32 + lane) * 4) =
                        make_float4(acc[h][t][0], acc[h][t][1], acc[h][t][2], acc[h][t][3]);
        __syncthreads();
        for (int i = tid; i < M * 32; i += kThreads) {
            const int r = i & 31, m = i >> 5, n = first + r, h = r >> 4;
            if (n >= n1) continue;
            // row r & 15, column m & 7 of token tile m / 8: lane 4 (r & 7) + (m & 7) / 2, element 2 (r / 8 & 1) + (m & 1)
            const int at_lane = 4 * (r & 7) + ((m & 7) >> 1), elem = 2 * ((r >> 3) & 1) + (m & 1);
            const float* src = red + ((h * NT + (m >> 3)) * 32 + at_lane) * 4 + elem;
            float z = 0.0f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) z += src[q * 2 * NT * 128];
            const size_t at = static_cast<size_t>(m) * p.N + n;
            if (p.r.bias) z += Act<ACT>::to_f(reinterpret_cast<const T*>(p.r.bias)[n]);
            if (p.r.pre) reinterpret_cast<T*>(p.r.pre)[at] = Act<ACT>::from_f(z);
            z = fn_value(p.r.fn, z);
            if (p.r.residual) z += Act<ACT>::to_f(reinterpret_cast<const T*>(p.r.residual)[at]);
            static_cast<T*>(p.r.out)[at] = Act<ACT>::from_f(z);
        }
    }
    cp_async_wait_all();
}

template <int ACT, int NT> int launch_nt(const DenseRowsParams& p, int sms, const RaggedArgs& g) {
    constexpr int smem = RowsStage<NT>::SMEM;
    static PerDevice configured;
    const int rc = raise_smem_limit(configured, reinterpret_cast<const void*>(dense_rows_kernel<ACT, NT>), smem);
    if (rc != MOE_OK) return rc;
    const cudaError_t e =
        launch_pdl(dense_rows_kernel<ACT, NT>, dim3(sms < p.N ? sms : p.N), kThreads, smem, g.st, p);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", g.who, cudaGetErrorString(e));
    count_launch();
    return check_launch(g.who);
}

template <int ACT> int launch_act(const DenseRowsParams& p, int sms, const RaggedArgs& g) {
    if (p.M <= 8) return launch_nt<ACT, 1>(p, sms, g);
    if (p.M <= 16) return launch_nt<ACT, 2>(p, sms, g);
    return launch_nt<ACT, 4>(p, sms, g);
}

}  // namespace

int launch_dense_rows(const RaggedArgs& g) {
    const int sms = sm_count();
    if (sms <= 0) return fail(MOE_ERR_CUDA, "%s: no CUDA device", g.who);
    const DenseRowsParams p{static_cast<const uint16_t*>(g.a), static_cast<const uint16_t*>(g.w), g.p.rows, g.N, g.K,
                            (g.K + 63) / 64, g.p};
    return g.act == MOE_ACT_BF16 ? launch_act<MOE_ACT_BF16>(p, sms, g) : launch_act<MOE_ACT_F16>(p, sms, g);
}

}  // namespace moe
