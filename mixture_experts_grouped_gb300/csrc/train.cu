// Row operators of a training step: SwiGLU and its gradient, the gradient of a
// dense product's bias and activation, rows to the experts and the gradients of
// combine and routing. All are bound by HBM, or by a launch where there are few rows.
#include "fn.cuh"

namespace moe {
namespace {

// ---- SwiGLU ---------------------------------------------------------------------
//
//   h = g s u,   s = 1 / (1 + exp(-g));   d_u = d_h g s,   d_g = d_h u s (1 + g (1 - s))
//
// of [rows, 2 I] gate/up products (gate columns, then up). Each thread takes 16-byte
// vectors of 8 columns, numbered through over all rows; the threads that an SM holds keep
// enough loads in flight. Measured, 8192 x 14336: 100 us forward, 203 back with h given
// again, both 7.0 TB/s (the copy rate); 64 x 768: 1.4 us, a launch's latency.
constexpr int kGluThreads = 256;

template <int ACT, typename Index>
__global__ void __launch_bounds__(kGluThreads)
swiglu_kernel(const uint4* __restrict__ gu, uint4* __restrict__ h, Index vectors, Index V) {
    pdl_wait();
    const Index i = static_cast<Index>(blockIdx.x) * kGluThreads + threadIdx.x;
    if (i >= vectors) return;
    const Index r = i / V;
    const uint4* row = gu + static_cast<size_t>(i) + static_cast<size_t>(r) * V;
    float g[8], u[8], o[8];
    const uint4 gv = row[0], uv = row[V];
    unpack8<ACT>(gv, g);
    unpack8<ACT>(uv, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = silu_part(g[j], sigmoid_fast(g[j])) * u[j];
    h[i] = pack8<ACT>(o);
}

template <int ACT, typename Index>
__global__ void __launch_bounds__(kGluThreads)
swiglu_backward_kernel(const uint4* gu, const uint4* dh, uint4* dgu, uint4* h, Index vectors, Index V) {
    pdl_wait();
    const Index i = static_cast<Index>(blockIdx.x) * kGluThreads + threadIdx.x;
    if (i >= vectors) return;
    const Index r = i / V;
    const size_t at = static_cast<size_t>(i) + static_cast<size_t>(r) * V;
    float g[8], u[8], d[8], dg[8], du[8], o[8];
    const uint4 gv = gu[at], uv = gu[at + V], dv = dh[i];
    unpack8<ACT>(gv, g);
    unpack8<ACT>(uv, u);
    unpack8<ACT>(dv, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float s = sigmoid_fast(g[j]);
        const float f = silu_part(g[j], s);
        o[j] = f * u[j];
        du[j] = d[j] * f;
        dg[j] = d[j] * u[j] * silu_slope(g[j], s);
    }
    dgu[at] = pack8<ACT>(dg);
    dgu[at + V] = pack8<ACT>(du);
    if (h) h[i] = pack8<ACT>(o);
}

// ---- gradient of bias and activation ------------------------------------------------
//
//   dz = d_out f'(pre),   d_bias[n] = sum_m dz[m, n]
//
// A CTA takes 8 TX columns (TX threads across) and every C-th group of 256 / TX rows of a
// cluster of C CTAs; column sums are added over the CTA's rows of threads and then over
// the cluster in rank order (distributed shared memory), so no workspace is needed and
// the order depends on the sizes alone. TX = 32 where that fills the GPU, since HBM is kinder
// to 512 bytes of a row than to 128 (4096 x 14336, relu: 59 us, 69 with TX = 8), else 8 (1333 x
// 2816: relu 7.6 us, gelu 10, of 3.4 for the bytes). gelu takes 29 instructions an element where
// relu takes 13 (4096 x 14336: 83 us, issue slots 67% busy, and 41): with some 21 warps an SM
// its arithmetic and its loads overlap in part only.
constexpr int kBiasThreads = 256;

template <int ACT, int FN, int TX>
__global__ void __launch_bounds__(kBiasThreads, 4)  // (with three CTAs an SM, clusters of 8 left SMs empty)
bias_act_backward_kernel(const uint16_t* d_out, const uint16_t* pre, int M, int N, uint16_t* d_pre,
                         float* d_bias, int accumulate, int C) {
    pdl_wait();
    constexpr int kBiasCols = 8 * TX, kBiasRows = kBiasThreads / TX;
    __shared__ float part[kBiasRows][kBiasCols];
    __shared__ float total[kBiasCols];
    const int tid = threadIdx.x, cv = tid % TX, ty = tid / TX;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n = blockIdx.x / C * kBiasCols + cv * 8;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    if (n < N) {
        // rows whose loads are in flight together (d_pre may be d_out or pre: the compiler would not)
        constexpr int BATCH = 4;
        const int stride = C * kBiasRows;
        for (int m0 = rank * kBiasRows + ty; m0 < M; m0 += BATCH * stride) {
            uint4 dv[BATCH], zv[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const size_t at = static_cast<size_t>(m0 + i * stride) * N + n;
                dv[i] = zv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (m0 + i * stride < M) {
                    dv[i] = *reinterpret_cast<const uint4*>(d_out + at);
                    if (FN != MOE_FN_NONE) zv[i] = *reinterpret_cast<const uint4*>(pre + at);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (m0 + i * stride >= M) break;
                float d[8], z[8];
                unpack8<ACT>(dv[i], d);
                if (FN != MOE_FN_NONE) {
                    unpack8<ACT>(zv[i], z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = __fmul_rn(d[j], fn_slope(FN, z[j]));  // (not fused with the sum)
                }
                if (d_pre)
                    *reinterpret_cast<uint4*>(d_pre + static_cast<size_t>(m0 + i * stride) * N + n) = pack8<ACT>(d);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += d[j];
            }
        }
    }
    if (!d_bias) return;  // (uniform: no CTA of the cluster waits)
#pragma unroll
    for (int j = 0; j < 8; ++j) part[ty][cv * 8 + j] = acc[j];
    __syncthreads();
    if (tid < kBiasCols) {
        float v = 0.0f;
#pragma unroll
        for (int r = 0; r < kBiasRows; ++r) v += part[r][tid];
        total[tid] = v;
    }
    if (C > 1) {
        __syncthreads();
        cluster_sync_all();
        if (rank == 0 && tid < kBiasCols) {
            float v = 0.0f;
            for (int r = 0; r < C; ++r) v += ld_dsmem_f32(mapa_shared(smem_u32(&total[tid]), r));
            total[tid] = v;
        }
        __syncwarp();
        cluster_sync_all();  // no CTA leaves before its sums are read
    }
    const int col = blockIdx.x / C * kBiasCols + tid;
    if (rank == 0 && tid < kBiasCols && col < N) d_bias[col] = accumulate ? d_bias[col] + total[tid] : total[tid];
}

// ---- rows to the experts, gradient of the combine -----------------------------------
//
// A block takes one token and 8 columns a thread at a time: its row is read once and
// serves the token's K rows, whose accesses are all in flight together. Bound by HBM, at
// rows in random order: 4096 tokens of 4096 columns, k = 2, 18.7 and 29.7 us, 5.4 and 5.7
// TB/s; 61 of 2048, k = 8, 3.5 and 3.8 us (row numbers, rows, stores, one after the other).
template <int K>
__global__ void __launch_bounds__(256)
dispatch_kernel(const uint4* x, const int32_t* __restrict__ pair_to_row, uint4* xs, int T, int V, int top_k,
                int max_rows, int32_t* err) {
    pdl_wait();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int row[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            row[j] = j < top_k ? __ldg(pair_to_row + t * top_k + j) : -1;
            if (row[j] >= max_rows) {
                if (threadIdx.x == 0) set_err(err, MOE_DEV_ERR_PAIR_ID);
                row[j] = -1;
            }
        }
        for (int v = threadIdx.x; v < V; v += blockDim.x) {
            const uint4 a = x[t * V + v];
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (row[j] >= 0) xs[static_cast<size_t>(row[j]) * V + v] = a;
        }
    }
}

template <int ACT, int K>
__global__ void __launch_bounds__(256)
combine_backward_kernel(const uint4* d_out, const uint4* y, const int32_t* __restrict__ pair_to_row,
                        const float* __restrict__ w, uint4* d_y, float* d_w, int T, int V, int top_k, int max_rows,
                        int32_t* err) {
    pdl_wait();
    __shared__ float part[8][K];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int row[K];
        float wt[K], acc[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            row[j] = j < top_k ? __ldg(pair_to_row + t * top_k + j) : -1;
            wt[j] = j < top_k ? __ldg(w + t * top_k + j) : 0.0f;
            acc[j] = 0.0f;
            if (row[j] >= max_rows) {
                if (tid == 0) set_err(err, MOE_DEV_ERR_PAIR_ID);
                row[j] = -1;
            }
        }
        for (int v = tid; v < V; v += blockDim.x) {
            float d[8];
            unpack8<ACT>(d_out[t * V + v], d);
            uint4 yv[K];
#pragma unroll
            for (int j = 0; j < K; ++j)
                yv[j] = row[j] >= 0 ? y[static_cast<size_t>(row[j]) * V + v] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (row[j] < 0) continue;
                float f[8], o[8];
                unpack8<ACT>(yv[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[j] = fmaf(d[i], f[i], acc[j]);
                    o[i] = wt[j] * d[i];
                }
                d_y[static_cast<size_t>(row[j]) * V + v] = pack8<ACT>(o);
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
            if (lane == 0) part[warp][j] = acc[j];
        }
        __syncthreads();
        if (tid < top_k) {
            float v = 0.0f;
            for (int i = 0; i < warps; ++i) v += part[i][tid];
            d_w[t * top_k + tid] = v;
        }
        __syncthreads();
    }
}

// ---- gradient of the routing: a warp a row -------------------------------------------
// 61 rows of 128 experts 3.8 us, 4096 of 8 3.7: latency.
__global__ void __launch_bounds__(128)
route_backward_kernel(const float* logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
                      const float* __restrict__ dw, float* dl, int T, int E, int top_k, int renorm, int32_t* err) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (t >= T) return;
    constexpr int PER = MOE_MAX_EXPERTS / 32;
    float p[PER];
    int id = -1;
    float wj = 0.0f, dj = 0.0f;
    // (every load at once: a row is bound by their latency)
    if (lane < top_k) {
        id = ids[t * top_k + lane];
        wj = w[t * top_k + lane];
        dj = dw[t * top_k + lane];
    }
    if (!renorm)
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] = lane + 32 * j < E ? logits[t * E + lane + 32 * j] : -INFINITY;
    if (lane < top_k && (id < 0 || id >= E)) {
        set_err(err, MOE_DEV_ERR_EXPERT_ID);
        id = -1;
        wj = dj = 0.0f;
    }
    float m = wj * dj;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m += __shfl_xor_sync(0xffffffffu, m, off);
    float scale = 1.0f;  // p times it is the softmax
    if (!renorm) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) top = fmaxf(top, p[j]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (32 * j >= E) break;
            p[j] = lane + 32 * j < E ? expf(p[j] - top) : 0.0f;
            sum += p[j];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        scale = __fdiv_rn(1.0f, sum);
    }
    // renormalised: what a slot gives its expert; otherwise the slot's part of g
    const float mine = renorm ? wj * (dj - m) : dj;
    float g[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) g[j] = 0.0f;
    for (int s = 0; s < top_k; ++s) {
        const int e = __shfl_sync(0xffffffffu, id, s);
        const float v = __shfl_sync(0xffffffffu, mine, s);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (32 * j >= E) break;
            if (e == lane + 32 * j) g[j] += v;
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (32 * j >= E) break;
        if (lane + 32 * j < E) dl[t * E + lane + 32 * j] = renorm ? g[j] : p[j] * scale * (g[j] - m);
    }
}

// ---- launches ------------------------------------------------------------------------

template <typename F> cudaError_t by_act(int act, F f) {
    return act == MOE_ACT_BF16 ? f(std::integral_constant<int, MOE_ACT_BF16>{})
                               : f(std::integral_constant<int, MOE_ACT_F16>{});
}
// the power of two that holds top_k
template <typename F> cudaError_t by_top_k(int top_k, F f) {
    if (top_k <= 1) return f(std::integral_constant<int, 1>{});
    if (top_k <= 2) return f(std::integral_constant<int, 2>{});
    if (top_k <= 4) return f(std::integral_constant<int, 4>{});
    if (top_k <= 8) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

int done(const char* who, cudaError_t e) {
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    count_launch();
    return check_launch(who);
}

// threads for rows of V vectors
int row_threads(int V) { return V >= 256 ? 256 : (V + 31) / 32 * 32; }

}  // namespace
}  // namespace moe

#define MOE_REQUIRE_ACT(act) \
    MOE_REQUIRE((act) == MOE_ACT_BF16 || (act) == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act)

extern "C" int moe_swiglu(const void* gate_up, int32_t act, int32_t rows, int32_t I, void* h, void* stream) {
    const char* who = "moe_swiglu";
    MOE_REQUIRE_ACT(act);
    MOE_REQUIRE(rows >= 0, "%s: rows=%d is negative", who, rows);
    MOE_REQUIRE(I > 0 && I % 8 == 0, "%s: I=%d must be a positive multiple of 8", who, I);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(gate_up && h, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(gate_up) && moe::aligned16(h), "%s: gate_up / h must be 16-byte aligned", who);
    const int64_t vectors = static_cast<int64_t>(rows) * (I / 8);
    const int64_t blocks = (vectors + moe::kGluThreads - 1) / moe::kGluThreads;
    if (blocks > 0x7fffffff) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: rows=%d x I=%d is too large", who, rows, I);
    const uint4* gu = static_cast<const uint4*>(gate_up);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return moe::done(who, moe::by_act(act, [&](auto a) {
        constexpr int A = decltype(a)::value;
        const dim3 grid(static_cast<unsigned>(blocks));
        if (vectors < (1u << 31))
            return moe::launch_pdl(moe::swiglu_kernel<A, uint32_t>, grid, moe::kGluThreads, 0, st, gu,
                                   static_cast<uint4*>(h), static_cast<uint32_t>(vectors), static_cast<uint32_t>(I / 8));
        return moe::launch_pdl(moe::swiglu_kernel<A, uint64_t>, grid, moe::kGluThreads, 0, st, gu,
                               static_cast<uint4*>(h), static_cast<uint64_t>(vectors), static_cast<uint64_t>(I / 8));
    }));
}

extern "C" int moe_swiglu_backward(const void* gate_up, const void* d_h, int32_t act, int32_t rows, int32_t I,
                                   void* d_gate_up, void* h, void* stream) {
    const char* who = "moe_swiglu_backward";
    MOE_REQUIRE_ACT(act);
    MOE_REQUIRE(rows >= 0, "%s: rows=%d is negative", who, rows);
    MOE_REQUIRE(I > 0 && I % 8 == 0, "%s: I=%d must be a positive multiple of 8", who, I);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(gate_up && d_h && d_gate_up, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(gate_up) && moe::aligned16(d_h) && moe::aligned16(d_gate_up) && moe::aligned16(h),
                "%s: tensors must be 16-byte aligned", who);
    const int64_t vectors = static_cast<int64_t>(rows) * (I / 8);
    const int64_t blocks = (vectors + moe::kGluThreads - 1) / moe::kGluThreads;
    if (blocks > 0x7fffffff) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: rows=%d x I=%d is too large", who, rows, I);
    const uint4 *gu = static_cast<const uint4*>(gate_up), *dh = static_cast<const uint4*>(d_h);
    uint4 *dgu = static_cast<uint4*>(d_gate_up), *hv = static_cast<uint4*>(h);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return moe::done(who, moe::by_act(act, [&](auto a) {
        constexpr int A = decltype(a)::value;
        const dim3 grid(static_cast<unsigned>(blocks));
        if (vectors < (1u << 31))
            return moe::launch_pdl(moe::swiglu_backward_kernel<A, uint32_t>, grid, moe::kGluThreads, 0, st, gu, dh, dgu,
                                   hv, static_cast<uint32_t>(vectors), static_cast<uint32_t>(I / 8));
        return moe::launch_pdl(moe::swiglu_backward_kernel<A, uint64_t>, grid, moe::kGluThreads, 0, st, gu, dh, dgu, hv,
                               static_cast<uint64_t>(vectors), static_cast<uint64_t>(I / 8));
    }));
}

extern "C" int moe_bias_act_backward(const void* d_out, const void* pre, int32_t act, int32_t fn, int32_t M, int32_t N,
                                     void* d_pre, float* d_bias, int32_t accumulate, void* stream) {
    const char* who = "moe_bias_act_backward";
    MOE_REQUIRE_ACT(act);
    MOE_REQUIRE(fn >= MOE_FN_NONE && fn <= MOE_FN_SILU, "%s: unknown activation function %d", who, fn);
    MOE_REQUIRE(M >= 0, "%s: M=%d is negative", who, M);
    MOE_REQUIRE(N > 0 && N % 8 == 0, "%s: N=%d must be a positive multiple of 8", who, N);
    if (M > (1 << 30)) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: M=%d above 2^30", who, M);
    MOE_REQUIRE(d_pre || d_bias, "%s: neither d_pre nor d_bias is given", who);
    MOE_REQUIRE(M == 0 || (d_out && (pre || fn == MOE_FN_NONE)), "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(d_out) && moe::aligned16(pre) && moe::aligned16(d_pre) && moe::aligned16(d_bias),
                "%s: tensors must be 16-byte aligned", who);
    if (M == 0 && !d_bias) return MOE_OK;  // (of no rows the bias' gradient is 0, and is written)
    // as many CTAs share a column tile as it has groups of rows, 8 at most
    const bool wide = (static_cast<int64_t>(N) + 255) / 256 * 8 >= 2 * moe::sm_count() && M >= 256;
    const int rows = wide ? 8 : 32, cols = wide ? 256 : 64;
    int C = 1;
    while (C < 8 && C * rows < M) C *= 2;
    const int64_t blocks = (static_cast<int64_t>(N) + cols - 1) / cols * C;
    if (blocks > 0x7fffffff) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: N=%d is too large", who, N);
    return moe::done(who, moe::by_act(act, [&](auto a) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = C;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(blocks));
        cfg.blockDim = dim3(moe::kBiasThreads);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cfg.attrs = attr;
        cfg.numAttrs = C > 1 ? 2 : 1;
        constexpr int A = decltype(a)::value;
        auto run = [&](auto f) {
            constexpr int F = decltype(f)::value;
            return cudaLaunchKernelEx(&cfg,
                                      wide ? moe::bias_act_backward_kernel<A, F, 32>
                                           : moe::bias_act_backward_kernel<A, F, 8>,
                                      static_cast<const uint16_t*>(d_out), static_cast<const uint16_t*>(pre), M, N,
                                      static_cast<uint16_t*>(d_pre), d_bias, accumulate, C);
        };
        switch (fn) {
            case MOE_FN_RELU: return run(std::integral_constant<int, MOE_FN_RELU>{});
            case MOE_FN_GELU: return run(std::integral_constant<int, MOE_FN_GELU>{});
            case MOE_FN_GELU_TANH: return run(std::integral_constant<int, MOE_FN_GELU_TANH>{});
            case MOE_FN_SILU: return run(std::integral_constant<int, MOE_FN_SILU>{});
            default: return run(std::integral_constant<int, MOE_FN_NONE>{});
        }
    }));
}

extern "C" int moe_dispatch(const void* x, int32_t act, const int32_t* pair_to_row, void* xs, int32_t T, int32_t H,
                            int32_t top_k, int32_t max_rows, int32_t* err_word, void* stream) {
    const char* who = "moe_dispatch";
    MOE_REQUIRE_ACT(act);
    MOE_REQUIRE(T >= 0 && max_rows >= 0, "%s: T=%d or max_rows=%d is negative", who, T, max_rows);
    MOE_REQUIRE(H > 0 && H % 8 == 0, "%s: H=%d must be a positive multiple of 8", who, H);
    MOE_REQUIRE(top_k >= 1 && top_k <= MOE_MAX_TOPK, "%s: top_k=%d outside [1, %d]", who, top_k, MOE_MAX_TOPK);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && pair_to_row && (xs || max_rows == 0), "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(x) && moe::aligned16(xs), "%s: x / xs must be 16-byte aligned", who);
    const int V = H / 8;
    return moe::done(who, moe::by_top_k(top_k, [&](auto k) {
        return moe::launch_pdl(moe::dispatch_kernel<decltype(k)::value>, dim3(T), moe::row_threads(V), 0,
                               static_cast<cudaStream_t>(stream), static_cast<const uint4*>(x), pair_to_row,
                               static_cast<uint4*>(xs), T, V, top_k, max_rows, err_word);
    }));
}

extern "C" int moe_combine_backward(const void* d_out, const void* y, int32_t act, const int32_t* pair_to_row,
                                    const float* topk_weights, void* d_y, float* d_weights, int32_t T, int32_t H,
                                    int32_t top_k, int32_t max_rows, int32_t* err_word, void* stream) {
    const char* who = "moe_combine_backward";
    MOE_REQUIRE_ACT(act);
    MOE_REQUIRE(T >= 0 && max_rows >= 0, "%s: T=%d or max_rows=%d is negative", who, T, max_rows);
    MOE_REQUIRE(H > 0 && H % 8 == 0, "%s: H=%d must be a positive multiple of 8", who, H);
    MOE_REQUIRE(top_k >= 1 && top_k <= MOE_MAX_TOPK, "%s: top_k=%d outside [1, %d]", who, top_k, MOE_MAX_TOPK);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(d_out && pair_to_row && topk_weights && d_weights && ((y && d_y) || max_rows == 0), "%s: NULL pointer",
                who);
    MOE_REQUIRE(moe::aligned16(d_out) && moe::aligned16(y) && moe::aligned16(d_y),
                "%s: d_out / y / d_y must be 16-byte aligned", who);
    const int V = H / 8;
    return moe::done(who, moe::by_act(act, [&](auto a) {
        return moe::by_top_k(top_k, [&](auto k) {
            return moe::launch_pdl(moe::combine_backward_kernel<decltype(a)::value, decltype(k)::value>, dim3(T),
                                   moe::row_threads(V), 0, static_cast<cudaStream_t>(stream),
                                   static_cast<const uint4*>(d_out), static_cast<const uint4*>(y), pair_to_row,
                                   topk_weights, static_cast<uint4*>(d_y), d_weights, T, V, top_k, max_rows, err_word);
        });
    }));
}

extern "C" int moe_route_backward(const float* logits, const int32_t* topk_ids, const float* topk_weights,
                                  const float* d_weights, float* d_logits, int32_t T, int32_t E, int32_t top_k,
                                  int32_t renormalize, int32_t* err_word, void* stream) {
    const char* who = "moe_route_backward";
    MOE_REQUIRE(E >= 1 && E <= MOE_MAX_EXPERTS, "%s: E=%d outside [1, %d]", who, E, MOE_MAX_EXPERTS);
    MOE_REQUIRE(top_k >= 1 && top_k <= E && top_k <= MOE_MAX_TOPK, "%s: top_k=%d outside [1, min(%d, %d)]", who, top_k, E,
                MOE_MAX_TOPK);
    MOE_REQUIRE(T >= 0, "%s: T=%d is negative", who, T);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(topk_ids && topk_weights && d_weights && d_logits && (logits || renormalize), "%s: NULL pointer", who);
    return moe::done(who, moe::launch_pdl(moe::route_backward_kernel, dim3((static_cast<unsigned>(T) + 3) / 4), 128, 0,
                                          static_cast<cudaStream_t>(stream), logits, topk_ids, topk_weights, d_weights,
                                          d_logits, T, E, top_k, renormalize, err_word));
}
