// Weight-streaming products for a few tokens: 16 weight rows against up to 8
// tokens at a time on warp-level tensor-core products (m16n8k16, 16-bit
// operands, f32 accumulation), the weights read from global memory straight
// into the fragments.
//
// With few tokens a product is bound by the weight bytes, so what matters is
// that every weight byte is loaded once, wide, with many loads in flight. The
// contraction index of a fragment is only a label: as long as both operands
// use the same order, a lane may take any k. Lane (g, c) = (lane / 4, lane % 4)
// therefore loads 16 consecutive bytes of rows g and g + 8, and the products
// of those bytes use them as their (2c, 2c + 1) and (2c + 8, 2c + 9) slots; the
// token operand loads the same k range of token g. No shared memory and no
// shuffles stand between HBM and the tensor core.
//
// A "unit" is what a warp takes at a time: 16 rows x SPAN contraction indices
// (one 16-byte load per row and lane). It is loaded into registers a ring
// ahead of its use.
#pragma once

#include "gemm_dequant.cuh"
#include "quant.cuh"

namespace moe {

__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldg_stream4(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

template <int ACT>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    if (ACT == MOE_ACT_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four E4M3 codes -> two words of two 16-bit values (exact in f16 and in bf16)
template <int ACT> __device__ __forceinline__ void e4m3x4_to_act(uint32_t w, uint32_t& p01, uint32_t& p23) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(p01), "=r"(p23)
        : "r"(w));
    if (ACT == MOE_ACT_BF16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&p01));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&p23));
        p01 = Act<MOE_ACT_BF16>::pack2(a.x, a.y);
        p23 = Act<MOE_ACT_BF16>::pack2(b.x, b.y);
    }
}

// One expert's weight [N, K] in global memory (see MoeWeight).
struct WBase {
    const uint8_t* w;
    const uint8_t* sc;
    const uint8_t* z;
    int N, K, G;
};

template <int FMT>
__device__ __forceinline__ WBase expert_base(const void* w, const void* sc, const void* z, int N, int K, int G,
                                             int e) {
    WBase b{static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(sc), static_cast<const uint8_t*>(z), N, K, G};
    const size_t nk = static_cast<size_t>(N) * K * e;
    if (FMT == MOE_W_BF16) b.w += nk * 2;
    if (FMT == MOE_W_FP8_E4M3) {
        b.w += nk;
        b.sc += static_cast<size_t>(N) * e * 4;
    }
    if (FMT == MOE_W_NVFP4) {
        b.w += nk / 2;
        b.sc += nk / 16;
    }
    if (FMT == MOE_W_GPTQ_INT4) {
        const size_t ng = static_cast<size_t>(K / G) * N * e;
        b.w += nk / 2;
        b.sc += ng * 2;
        b.z += ng / 2;
    }
    return b;
}

// Unit<FMT, ACT>: SPAN contraction indices of rows r0 and r1 (-1: no row, zeros).
//   CHUNKS     pieces of 8 contraction indices a lane holds per row
//   k_of(i)    contraction index of piece i, relative to the unit's first
//   frag(i)    piece i of both rows as A-operand words a0..a3 of two products
//   X_PERM     the token operand's 8 values go in the order 0,4,1,5,2,6,3,7
//   GROUPED    the unit's sums carry their own row scales s0 / s1 and are
//              scaled before they are added (otherwise row scales, if any,
//              multiply the finished sums)
template <int FMT, int ACT> struct Unit;

template <int ACT> struct Unit<MOE_W_BF16, ACT> {
    static constexpr int SPAN = 32, CHUNKS = 1;
    static constexpr bool X_PERM = false, GROUPED = false, ROW_SCALE = false;
    uint4 r[2];
    __device__ __forceinline__ void load(const WBase& b, int r0, int r1, int k0, int c) {
        const int k = k0 + 8 * c;
        const bool in = k < b.K;
        r[0] = (in && r0 >= 0) ? ldg_stream16(b.w + (static_cast<size_t>(r0) * b.K + k) * 2) : make_uint4(0, 0, 0, 0);
        r[1] = (in && r1 >= 0) ? ldg_stream16(b.w + (static_cast<size_t>(r1) * b.K + k) * 2) : make_uint4(0, 0, 0, 0);
    }
    static __device__ __forceinline__ int k_of(int, int c) { return 8 * c; }
    __device__ __forceinline__ void frag(int, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        a[0] = r[0].x; a[1] = r[0].y; a[2] = r[0].z; a[3] = r[0].w;
        b[0] = r[1].x; b[1] = r[1].y; b[2] = r[1].z; b[3] = r[1].w;
    }
    __device__ __forceinline__ float scale(int) const { return 1.0f; }
};

template <int ACT> struct Unit<MOE_W_FP8_E4M3, ACT> {
    static constexpr int SPAN = 64, CHUNKS = 2;
    static constexpr bool X_PERM = false, GROUPED = false, ROW_SCALE = true;
    uint4 r[2];
    float s[2];
    __device__ __forceinline__ void load(const WBase& b, int r0, int r1, int k0, int c) {
        const int k = k0 + 16 * c;
        const bool in = k < b.K;
        r[0] = (in && r0 >= 0) ? ldg_stream16(b.w + static_cast<size_t>(r0) * b.K + k) : make_uint4(0, 0, 0, 0);
        r[1] = (in && r1 >= 0) ? ldg_stream16(b.w + static_cast<size_t>(r1) * b.K + k) : make_uint4(0, 0, 0, 0);
        s[0] = r0 >= 0 ? __ldg(reinterpret_cast<const float*>(b.sc) + r0) : 0.0f;
        s[1] = r1 >= 0 ? __ldg(reinterpret_cast<const float*>(b.sc) + r1) : 0.0f;
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 16 * c + 8 * i; }
    __device__ __forceinline__ void frag(int i, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        e4m3x4_to_act<ACT>(i ? r[0].z : r[0].x, a[0], a[1]);
        e4m3x4_to_act<ACT>(i ? r[0].w : r[0].y, a[2], a[3]);
        e4m3x4_to_act<ACT>(i ? r[1].z : r[1].x, b[0], b[1]);
        e4m3x4_to_act<ACT>(i ? r[1].w : r[1].y, b[2], b[3]);
    }
    __device__ __forceinline__ float scale(int i) const { return s[i]; }
};

template <int ACT> struct Unit<MOE_W_NVFP4, ACT> {
    static constexpr int SPAN = 128, CHUNKS = 4;
    static constexpr bool X_PERM = false, GROUPED = false, ROW_SCALE = false;
    uint4 r[2];
    uint32_t sc[2];  // the two E4M3 block scales of the lane's 32 codes, low byte first
    __device__ __forceinline__ void load(const WBase& b, int r0, int r1, int k0, int c) {
        const int k = k0 + 32 * c;
        const bool in = k < b.K;
        const size_t sb = static_cast<size_t>(k / 16) * b.N;
        r[0] = r[1] = make_uint4(0, 0, 0, 0);
        sc[0] = sc[1] = 0;
        if (in && r0 >= 0) {
            r[0] = ldg_stream16(b.w + (static_cast<size_t>(r0) * b.K + k) / 2);
            sc[0] = __ldg(b.sc + sb + r0) | (static_cast<uint32_t>(__ldg(b.sc + sb + b.N + r0)) << 8);
        }
        if (in && r1 >= 0) {
            r[1] = ldg_stream16(b.w + (static_cast<size_t>(r1) * b.K + k) / 2);
            sc[1] = __ldg(b.sc + sb + r1) | (static_cast<uint32_t>(__ldg(b.sc + sb + b.N + r1)) << 8);
        }
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 32 * c + 8 * i; }
    static __device__ __forceinline__ void row(const uint4& w, uint32_t sc, int i, uint32_t (&o)[4]) {
        const uint32_t word = i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
        uint32_t s2[2];
        const uint32_t s[2] = {sc & 0xffu, sc >> 8};
        gemm::e4m3_scale_pairs<ACT, 2>(s, s2);
        const uint32_t m = s2[i >> 1];
        if (ACT == MOE_ACT_BF16) {
            gemm::e2m1x4_to_bf16x4(word, o[0], o[1]);
            gemm::e2m1x4_to_bf16x4(word >> 16, o[2], o[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o[j]),
                                                 *reinterpret_cast<const __nv_bfloat162*>(&m));
                o[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t e2 = gemm::e2m1x2_to_f16x2((word >> (8 * j)) & 0xffu);
                const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&e2), *reinterpret_cast<const __half2*>(&m));
                o[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
    }
    __device__ __forceinline__ void frag(int i, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        row(r[0], sc[0], i, a);
        row(r[1], sc[1], i, b);
    }
    __device__ __forceinline__ float scale(int) const { return 1.0f; }
};

// GPTQ: the words of 8 k values lie along n, so a lane loads single words. The
// fragments hold the integers q - z (exact), and the group's f16 scale
// multiplies the f32 sums of each unit: SPAN = 64 never crosses a group.
template <int ACT> struct Unit<MOE_W_GPTQ_INT4, ACT> {
    static constexpr int SPAN = 64, CHUNKS = 2;
    static constexpr bool X_PERM = true, GROUPED = true, ROW_SCALE = false;
    uint32_t w[2][2];  // [row][piece]
    uint32_t zw[2];    // the row's zero-point word, shifted to its nibble by frag
    uint16_t s[2];
    uint8_t sh[2];
    __device__ __forceinline__ void load1(const WBase& b, int q, int r, int k0, int c) {
        w[q][0] = w[q][1] = zw[q] = 0;
        s[q] = 0;
        sh[q] = static_cast<uint8_t>(4 * (r & 7));
        if (r < 0 || k0 >= b.K) return;
        const uint8_t* p = b.w + (static_cast<size_t>(k0 / 8 + c) * b.N + r) * 4;
        w[q][0] = ldg_stream4(p);
        w[q][1] = ldg_stream4(p + static_cast<size_t>(b.N) * 16);
        const size_t g = static_cast<size_t>(k0 / b.G);
        s[q] = __ldg(reinterpret_cast<const uint16_t*>(b.sc) + g * b.N + r);
        zw[q] = __ldg(reinterpret_cast<const uint32_t*>(b.z) + g * (b.N / 8) + r / 8);
    }
    __device__ __forceinline__ void load(const WBase& b, int r0, int r1, int k0, int c) {
        load1(b, 0, r0, k0, c);
        load1(b, 1, r1, k0, c);
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 8 * (c + 4 * i); }
    __device__ __forceinline__ void row(int q, int i, uint32_t (&o)[4]) const {
        const uint32_t z = (zw[q] >> sh[q]) & 15u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (k_j, k_{j+4})
            if (ACT == MOE_ACT_F16) {
                const uint32_t v = gemm::and_or(w[q][i] >> (4 * j), 0x000F000Fu, 0x64006400u);  // 1024 + q
                const __half2 zz = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6400u | z)));
                const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), zz);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            } else {
                const uint32_t v = gemm::and_or(w[q][i] >> (4 * j), 0x000F000Fu, 0x43004300u);  // 128 + q
                const __nv_bfloat162 zz =
                    __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(0x4300u | z)));
                const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), zz);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            }
        }
    }
    __device__ __forceinline__ void frag(int i, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        row(0, i, a);
        row(1, i, b);
    }
    __device__ __forceinline__ float scale(int q) const { return __half2float(__ushort_as_half(s[q])); }
};

// acc[tile] += unit x tokens, for nt tiles of 8 tokens. xp[tile] is the lane's
// token row (token g of the tile) or NULL (a zero operand), k0 the unit's first
// contraction index.
template <int FMT, int ACT, int NT>
__device__ __forceinline__ void unit_mma(const Unit<FMT, ACT>& u, const uint16_t* const (&xp)[NT], int nt, int k0,
                                         int K, int c, float (&acc)[NT][4]) {
    using U = Unit<FMT, ACT>;
    float part[NT][4];
    if (U::GROUPED) {
#pragma unroll
        for (int t = 0; t < NT; ++t) part[t][0] = part[t][1] = part[t][2] = part[t][3] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < U::CHUNKS; ++i) {
        const int k = k0 + U::k_of(i, c);
        uint32_t a[4], b[4];
        u.frag(i, a, b);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t < nt) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (xp[t] && k < K) x = *reinterpret_cast<const uint4*>(xp[t] + k);
                if (U::X_PERM)
                    x = make_uint4(gemm::prmt(x.x, x.z, 0x5410), gemm::prmt(x.x, x.z, 0x7632),
                                   gemm::prmt(x.y, x.w, 0x5410), gemm::prmt(x.y, x.w, 0x7632));
                float (&d)[4] = U::GROUPED ? part[t] : acc[t];
                mma_16816<ACT>(d, a[0], b[0], a[1], b[1], x.x, x.y);
                mma_16816<ACT>(d, a[2], b[2], a[3], b[3], x.z, x.w);
            }
        }
    }
    if (U::GROUPED) {
        const float s0 = u.scale(0), s1 = u.scale(1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t < nt) {
                acc[t][0] = fmaf(s0, part[t][0], acc[t][0]);
                acc[t][1] = fmaf(s0, part[t][1], acc[t][1]);
                acc[t][2] = fmaf(s1, part[t][2], acc[t][2]);
                acc[t][3] = fmaf(s1, part[t][3], acc[t][3]);
            }
        }
    }
}

}  // namespace moe
