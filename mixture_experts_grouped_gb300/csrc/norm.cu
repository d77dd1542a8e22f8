// Row operators of the serving path that end in E4M3 codes: residual addition
// with the root-mean-square norm, and SiLU-mul.
#include "quant.cuh"

namespace moe {
namespace {

// ---- residual addition + RMS norm (+ E4M3 output) -------------------------------
//
//   r = x + residual,  y = r * (1 / sqrt(mean(r^2) + eps)) * weight,
//   per 128 columns: s = max(amax |y| / 448, 2^-126), q = e4m3(y / s)
//
// Everything between the loads and the stores is f32 (r is not rounded before
// it is normed, y not before it is quantised). HBM-bound: a row is read once
// into registers (VPT 16-byte vectors a thread), its sum of squares reduced,
// and every output written from there. A group of 128 columns is half a warp,
// so its maximum takes four shuffles and no shared memory. Measured: 4001 rows
// of 4096, every output: 24.2 us, 6.1 TB/s; one row of 2048: 1.6 us, a launch's
// latency.

template <int ACT, int VPT>
struct NormRow {
    float v[VPT][8];
    // r = x + residual of this thread's vectors; writes r; returns its sum of squares
    __device__ __forceinline__ float load(const uint4* x, const uint4* res, uint4* res_out, int V, int first,
                                          int step) {
        float ss = 0.0f;
        uint4 a[VPT], b[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * step;
            a[j] = i < V ? x[i] : make_uint4(0u, 0u, 0u, 0u);
            b[j] = (i < V && res) ? res[i] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * step;
            unpack8<ACT>(a[j], v[j]);
            if (res) {
                float f[8];
                unpack8<ACT>(b[j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[j][q] = __fadd_rn(v[j][q], f[q]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) ss = fmaf(v[j][q], v[j][q], ss);
            if (res_out && i < V) res_out[i] = pack8<ACT>(v[j]);
        }
        return ss;
    }
    __device__ __forceinline__ void store(float rstd, const uint4* w, uint4* y, uint2* q, float* s, int V, int first,
                                          int step, int lane) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * step;
            float wv[8];
            unpack8<ACT>(i < V ? w[i] : make_uint4(0u, 0u, 0u, 0u), wv);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] = v[j][k] * rstd * wv[k];
            if (y && i < V) y[i] = pack8<ACT>(v[j]);
            if (q) {
                // lanes past the row hold NaN or 0 (0 * rstd * 0): they stay out of the maximum
                const float sc = group_scale(amax_half_warp(i < V ? amax8(v[j]) : 0.0f, 0xffffffffu));
                if (i < V) {
                    q[i] = e4m3x8(v[j], sc);
                    if ((lane & (kQuantLanes - 1)) == 0) s[i / kQuantLanes] = sc;
                }
            }
        }
    }
};

struct NormParams {
    const uint4* x;
    const uint4* res;
    const uint4* w;
    uint4* res_out;
    uint4* y;
    uint2* q;
    float* s;
    float eps;
    int T, H;
};

__device__ __forceinline__ float rms_rstd(float ss, int H, float eps) {
    return rsqrtf(__fdiv_rn(ss, static_cast<float>(H)) + eps);
}

constexpr int kNormWarpRows = 4;

// rows of up to 256 columns: a warp each
template <int ACT>
__global__ void __launch_bounds__(32 * kNormWarpRows) add_rmsnorm_warp_kernel(const NormParams p) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kNormWarpRows + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int V = p.H / 8;
    const size_t row = static_cast<size_t>(t) * V;
    NormRow<ACT, 1> r;
    float ss = r.load(p.x + row, p.res ? p.res + row : nullptr, p.res_out ? p.res_out + row : nullptr, V, lane, 32);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const int groups = (p.H + kQuantGroup - 1) / kQuantGroup;
    r.store(rms_rstd(ss, p.H, p.eps), p.w, p.y ? p.y + row : nullptr, p.q ? p.q + row : nullptr,
            p.q ? p.s + static_cast<size_t>(t) * groups : nullptr, V, lane, 32, lane);
}

// longer rows: a block each
template <int ACT, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_block_kernel(const NormParams p) {
    pdl_wait();
    __shared__ float part[32];
    const int tid = threadIdx.x, lane = tid & 31, n = blockDim.x;
    const int t = blockIdx.x;
    const int V = p.H / 8;
    const size_t row = static_cast<size_t>(t) * V;
    NormRow<ACT, VPT> r;
    float ss = r.load(p.x + row, p.res ? p.res + row : nullptr, p.res_out ? p.res_out + row : nullptr, V, tid, n);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (lane == 0) part[tid >> 5] = ss;
    __syncthreads();
    ss = lane < (n >> 5) ? part[lane] : 0.0f;  // every warp adds the warps' sums in the same order
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const int groups = (p.H + kQuantGroup - 1) / kQuantGroup;
    r.store(rms_rstd(ss, p.H, p.eps), p.w, p.y ? p.y + row : nullptr, p.q ? p.q + row : nullptr,
            p.q ? p.s + static_cast<size_t>(t) * groups : nullptr, V, tid, n, lane);
}

// A row's form does not depend on how many rows there are, so neither do its
// bits. 262144 rows of 256 columns take 88 us a warp each, 134 a block; one row
// of 512 1.9 us a warp, 1.5 a block. One vector a thread keeps the most loads in
// flight (one row of 4096: 1.8 us, 2.2 with two vectors); above 1024 threads it
// is four (4096 rows of 16384: 97.8 us, 105 with two).
template <int ACT>
cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
    const int V = p.H / 8;
    if (V <= 32)
        return launch_pdl(add_rmsnorm_warp_kernel<ACT>, (p.T - 1) / kNormWarpRows + 1, 32 * kNormWarpRows, 0, st, p);
    if (V <= 1024) return launch_pdl(add_rmsnorm_block_kernel<ACT, 1>, p.T, (V + 31) / 32 * 32, 0, st, p);
    return launch_pdl(add_rmsnorm_block_kernel<ACT, 4>, p.T, ((V + 3) / 4 + 31) / 32 * 32, 0, st, p);
}

// ---- SiLU-mul with E4M3 output -----------------------------------------------------
//
//   v = g / (1 + exp(-g)) * u,  s = max(amax |v| / 448, 2^-126),  q = e4m3(v / s)
//
// of a [T, 2I] gate/up product (gate columns, then up). HBM-bound: 4 bytes in
// and 1 byte out per element of [T, I]. Each thread takes 8 columns, a half
// warp one group of 128; the groups of all rows are numbered through, so rows
// of any width fill the blocks. Two groups a half warp keep twice the loads in
// flight (T = 4096, I = 14336: 46.2 us, 6.4 TB/s; 56.4 with one group, 64-bit
// group numbers and the library's exponential and division, whose instructions
// bound it); a short last group leaves lanes idle (I = 136: 3.9 TB/s).
constexpr int kSiluThreads = 128;
constexpr int kSiluItems = 2;  // groups a half warp takes

template <int ACT, typename Index>
__global__ void __launch_bounds__(kSiluThreads)
silu_mul_quant_kernel(const uint4* __restrict__ gu, uint2* __restrict__ q, float* __restrict__ s, int T, int I) {
    pdl_wait();
    const int V = I / 8;                                        // vectors per row
    const Index groups = (I + kQuantGroup - 1) / kQuantGroup;
    const Index all = static_cast<Index>(T) * groups;
    const int lane = threadIdx.x & (kQuantLanes - 1);
    uint4 gv[kSiluItems], uv[kSiluItems];
    Index group[kSiluItems];
    size_t at[kSiluItems];  // vector of the output; V (of no row) where this lane has none
    bool in[kSiluItems];
#pragma unroll
    for (int j = 0; j < kSiluItems; ++j) {
        group[j] = (static_cast<Index>(blockIdx.x) * kSiluItems + j) * (kSiluThreads / kQuantLanes) +
                   threadIdx.x / kQuantLanes;
        const Index t = group[j] / groups;
        const int v = static_cast<int>(group[j] - t * groups) * kQuantLanes + lane;
        in[j] = group[j] < all && v < V;
        at[j] = static_cast<size_t>(t) * V + v;
        gv[j] = uv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (in[j]) {
            const uint4* row = gu + at[j] + static_cast<size_t>(t) * V;
            gv[j] = __ldcs(row);
            uv[j] = __ldcs(row + V);
        }
    }
#pragma unroll
    for (int j = 0; j < kSiluItems; ++j) {
        float g[8], u[8], o[8];
        unpack8<ACT>(gv[j], g);
        unpack8<ACT>(uv[j], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = silu_mul_fast(g[i], u[i]);
        // a lane past the row or the last group holds zeros, which stay out of the maximum
        const float sc = group_scale(amax_half_warp(amax8(o), 0xffffffffu));
        if (in[j]) {
            q[at[j]] = e4m3x8(o, sc);
            if (lane == 0) s[group[j]] = sc;
        }
    }
}

template <int ACT>
cudaError_t launch_silu(const uint4* gu, uint2* q, float* s, int T, int I, unsigned blocks, cudaStream_t st) {
    if (blocks < (1u << 27))  // the group numbers fit in 32 bits: their division is a few instructions, not a hundred
        return launch_pdl(silu_mul_quant_kernel<ACT, uint32_t>, dim3(blocks), kSiluThreads, 0, st, gu, q, s, T, I);
    return launch_pdl(silu_mul_quant_kernel<ACT, uint64_t>, dim3(blocks), kSiluThreads, 0, st, gu, q, s, T, I);
}

}  // namespace
}  // namespace moe

extern "C" int moe_add_rmsnorm_quant(const void* x, const void* residual, int32_t act, const void* weight, float eps,
                                     int32_t T, int32_t H, void* residual_out, void* y, void* q, float* q_scales,
                                     void* stream) {
    const char* who = "moe_add_rmsnorm_quant";
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(T >= 0, "%s: T=%d is negative", who, T);
    MOE_REQUIRE(H > 0 && H % 8 == 0, "%s: H=%d must be a positive multiple of 8", who, H);
    MOE_REQUIRE(eps >= 0.0f, "%s: eps=%g must not be negative", who, static_cast<double>(eps));
    if (H > MOE_MAX_NORM_H)
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: H=%d above %d", who, H, MOE_MAX_NORM_H);
    MOE_REQUIRE(y || q, "%s: neither y nor q is given", who);
    MOE_REQUIRE((q == nullptr) == (q_scales == nullptr), "%s: q and q_scales go together", who);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && weight, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(x) && moe::aligned16(residual) && moe::aligned16(weight) &&
                    moe::aligned16(residual_out) && moe::aligned16(y) && moe::aligned16(q),
                "%s: tensors must be 16-byte aligned", who);
    MOE_REQUIRE((reinterpret_cast<uintptr_t>(q_scales) & 3u) == 0, "%s: q_scales must be 4-byte aligned", who);
    const moe::NormParams p{static_cast<const uint4*>(x), static_cast<const uint4*>(residual),
                            static_cast<const uint4*>(weight), static_cast<uint4*>(residual_out),
                            static_cast<uint4*>(y), static_cast<uint2*>(q), q_scales, eps, T, H};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        act == MOE_ACT_BF16 ? moe::launch_norm<MOE_ACT_BF16>(p, st) : moe::launch_norm<MOE_ACT_F16>(p, st);
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch();
    return moe::check_launch(who);
}

extern "C" int moe_silu_mul_quant(const void* gate_up, int32_t act, int32_t T, int32_t I, void* q, float* q_scales,
                                  void* stream) {
    const char* who = "moe_silu_mul_quant";
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(T >= 0, "%s: T=%d is negative", who, T);
    MOE_REQUIRE(I > 0 && I % 8 == 0, "%s: I=%d must be a positive multiple of 8", who, I);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(gate_up && q && q_scales, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(gate_up) && moe::aligned16(q), "%s: gate_up / q must be 16-byte aligned", who);
    MOE_REQUIRE((reinterpret_cast<uintptr_t>(q_scales) & 3u) == 0, "%s: q_scales must be 4-byte aligned", who);
    const int64_t groups = static_cast<int64_t>(T) * ((I + moe::kQuantGroup - 1) / moe::kQuantGroup);
    constexpr int kPerBlock = moe::kSiluItems * moe::kSiluThreads / moe::kQuantLanes;
    const int64_t blocks = (groups + kPerBlock - 1) / kPerBlock;
    if (blocks > 0x7fffffff) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: T=%d x I=%d is too large", who, T, I);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint4* gu = static_cast<const uint4*>(gate_up);
    uint2* qv = static_cast<uint2*>(q);
    const unsigned grid = static_cast<unsigned>(blocks);
    const cudaError_t e = act == MOE_ACT_BF16 ? moe::launch_silu<MOE_ACT_BF16>(gu, qv, q_scales, T, I, grid, st)
                                              : moe::launch_silu<MOE_ACT_F16>(gu, qv, q_scales, T, I, grid, st);
    if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    moe::count_launch();
    return moe::check_launch(who);
}
