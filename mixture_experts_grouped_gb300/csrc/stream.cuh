// Weight-streaming products for a few tokens: 16 weight rows against up to 8
// tokens at a time on warp-level tensor-core products (m16n8k16, 16-bit
// operands, f32 accumulation).
//
// With few tokens a product is bound by the weight bytes, so what matters is
// that every weight byte is loaded once, in wide pieces, with enough of them
// in flight (about 40 KB per SM cover HBM's latency at its full rate) and few
// instructions per byte: at full rate an SM has 23 bytes per clock to digest,
// 4 issue slots each. The contraction index of a fragment is only a label: as
// long as both operands use the same order, a lane may take any k. Lane (g, c)
// = (lane / 4, lane % 4) therefore takes 16 consecutive bytes of rows g and
// g + 8, and the products use them as their (2c, 2c + 1) and (2c + 8, 2c + 9)
// slots; the token operand takes the same k range of token g.
//
// A "unit" is what a warp takes at a time: 16 rows x SPAN contraction indices.
// Units arrive by cp.async in a ring of shared-memory stages private to the
// warp. Each lane copies what it will itself read (only scales cross lanes),
// so a stage needs no barrier beyond the warp's own, and what is in flight
// takes no registers. (The same ring in registers ran at a fifth of HBM's
// rate: loads and conversions kept the ring's registers from staying in
// flight.)
#pragma once

#include "gemm_dequant.cuh"
#include "quant.cuh"

namespace moe {

__device__ __forceinline__ void cp_async4_zfill(void* dst, const void* src, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(full ? 4 : 0)
                 : "memory");
}
// 16 bytes through L1 (token operands: neighbouring warps and later tiles read them again)
__device__ __forceinline__ void cp_async16_l1(void* dst, const void* src, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(full ? 16 : 0)
                 : "memory");
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

// Two sets of up to 8 weight rows: a, a + 1, ... (lane groups g < na) and b, ... (g < nb).
struct UnitRows {
    int a, na, b, nb;
};

// Unit<FMT, ACT>: one format's stage layout and fragments.
//   SPAN       contraction indices per unit
//   CHUNKS     pieces of 8 contraction indices a lane holds per row
//   BYTES      weights and scales of a unit in a stage
//   X_RING     the first token tile's values ride in the stage too (formats
//              whose conversion is too short to hide their latency)
//   X_PERM     the token operand's 8 values go in the order 0,4,1,5,2,6,3,7
//   GROUPED    a unit's sums are scaled (row_scale) before they are added
//   Src        where a lane copies from: set to an expert's rows by aim(), then
//              load() copies the unit at contraction index k0
//   open       reads a stage's words and scales into registers
//   frag(i)    piece i of both rows as the A operands of two products
// Copies past the contraction's end are filled with zeros (the token operand
// too); a row past the unit's rows is not copied: it only feeds sums that
// nobody reads.
template <int FMT, int ACT> struct Unit;

// rows of K contiguous elements of EB bits, 16 bytes of each row and lane
template <int EB> struct RowSrc {
    const uint8_t* pa;
    const uint8_t* pb;
    bool va, vb;
    int kc;  // the lane's first contraction index within a unit
    __device__ __forceinline__ void aim(const WBase& b, const UnitRows& u, int lane) {
        const int g = lane >> 2;
        kc = (lane & 3) * (128 / EB);
        va = g < u.na;
        vb = g < u.nb;
        pa = b.w + (static_cast<size_t>(u.a + g) * b.K + kc) * EB / 8;
        pb = b.w + (static_cast<size_t>(u.b + g) * b.K + kc) * EB / 8;
    }
    __device__ __forceinline__ void load(uint8_t* st, int k0, int K, bool tail, int lane) const {
        const int off = k0 * EB / 8;
        if (!tail) {
            if (va) cp_async16(st + 16 * lane, pa + off);
            if (vb) cp_async16(st + 512 + 16 * lane, pb + off);
        } else {
            const bool in = k0 + kc < K;  // a skipped copy reads nothing, but its address stays the row's own
            if (va) cp_async16_zfill(st + 16 * lane, pa + (in ? off : 0), in);
            if (vb) cp_async16_zfill(st + 512 + 16 * lane, pb + (in ? off : 0), in);
        }
    }
};

template <int ACT> struct Unit<MOE_W_BF16, ACT> {
    static constexpr int SPAN = 32, CHUNKS = 1, BYTES = 1024;
    static constexpr bool X_RING = true, X_PERM = false, GROUPED = false, ROW_SCALE = false;
    struct Src : RowSrc<16> {};
    uint4 r[2];
    __device__ __forceinline__ void open(const uint8_t* st, const UnitRows&, int lane) {
        r[0] = *reinterpret_cast<const uint4*>(st + 16 * lane);
        r[1] = *reinterpret_cast<const uint4*>(st + 512 + 16 * lane);
    }
    static __device__ __forceinline__ int k_of(int, int c) { return 8 * c; }
    __device__ __forceinline__ void frag(int, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        a[0] = r[0].x; a[1] = r[0].y; a[2] = r[0].z; a[3] = r[0].w;
        b[0] = r[1].x; b[1] = r[1].y; b[2] = r[1].z; b[3] = r[1].w;
    }
    __device__ __forceinline__ float row_scale(int) const { return 1.0f; }
};

template <int ACT> struct Unit<MOE_W_FP8_E4M3, ACT> {
    static constexpr int SPAN = 64, CHUNKS = 2, BYTES = 1024;
    static constexpr bool X_RING = false, X_PERM = false, GROUPED = false, ROW_SCALE = true;
    struct Src : RowSrc<8> {};
    uint4 r[2];
    __device__ __forceinline__ void open(const uint8_t* st, const UnitRows&, int lane) {
        r[0] = *reinterpret_cast<const uint4*>(st + 16 * lane);
        r[1] = *reinterpret_cast<const uint4*>(st + 512 + 16 * lane);
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 16 * c + 8 * i; }
    __device__ __forceinline__ void frag(int i, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        e4m3x4_to_act<ACT>(i ? r[0].z : r[0].x, a[0], a[1]);
        e4m3x4_to_act<ACT>(i ? r[0].w : r[0].y, a[2], a[3]);
        e4m3x4_to_act<ACT>(i ? r[1].z : r[1].x, b[0], b[1]);
        e4m3x4_to_act<ACT>(i ? r[1].w : r[1].y, b[2], b[3]);
    }
    __device__ __forceinline__ float row_scale(int) const { return 1.0f; }
};

// NVFP4: the block scales lie along n, one byte each: a stage holds, for each
// row set and each of the unit's 8 blocks, the three aligned words around its
// 8 rows (48 words: one per lane, and a second for half the lanes).
template <int ACT> struct Unit<MOE_W_NVFP4, ACT> {
    static constexpr int SPAN = 128, CHUNKS = 4, BYTES = 1024 + 192;
    static constexpr bool X_RING = false, X_PERM = false, GROUPED = false, ROW_SCALE = false;
    struct Src : RowSrc<4> {
        const uint8_t* ps[2];
        int kb[2];  // block within the unit
        bool vs[2];
        int N;
        __device__ __forceinline__ void aim(const WBase& b, const UnitRows& u, int lane) {
            RowSrc<4>::aim(b, u, lane);
            N = b.N;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = lane + 32 * h, set = p / 24, q = p - 24 * set;
                const int n = ((set ? u.b : u.a) & ~3) + 4 * (q % 3);
                kb[h] = q / 3;
                vs[h] = p < 48 && n < b.N;
                ps[h] = b.sc + static_cast<size_t>(kb[h]) * b.N + n;
            }
        }
        __device__ __forceinline__ void load(uint8_t* st, int k0, int K, bool tail, int lane) const {
            RowSrc<4>::load(st, k0, K, tail, lane);
            const int off = (k0 >> 4) * N;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!vs[h]) continue;
                uint8_t* d = st + 1024 + 4 * lane + 128 * h;
                if (!tail) {
                    cp_async4(d, ps[h] + off);
                } else {  // a scale past the end meets zero codes, but must not be a NaN
                    const bool in = k0 + 16 * kb[h] < K;
                    cp_async4_zfill(d, ps[h] + (in ? off : -kb[h] * N), in);
                }
            }
        }
    };
    uint4 r[2];
    uint32_t sc[2];  // the two block scales of the lane's 32 codes, low byte first
    __device__ __forceinline__ void open(const uint8_t* st, const UnitRows& u, int lane) {
        const int g = lane >> 2, c = lane & 3;
        r[0] = *reinterpret_cast<const uint4*>(st + 16 * lane);
        r[1] = *reinterpret_cast<const uint4*>(st + 512 + 16 * lane);
        const uint8_t* s0 = st + 1024 + 24 * c + (u.a & 3) + g;
        const uint8_t* s1 = st + 1024 + 96 + 24 * c + (u.b & 3) + g;
        sc[0] = s0[0] | (static_cast<uint32_t>(s0[12]) << 8);
        sc[1] = s1[0] | (static_cast<uint32_t>(s1[12]) << 8);
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
    __device__ __forceinline__ float row_scale(int) const { return 1.0f; }
};

// GPTQ: the words of 8 k values lie along n, so a lane copies single words. The
// fragments hold the integers q - z (exact), and the group's f16 scale
// multiplies the f32 sums of each unit: SPAN = 64 divides every group. Per row
// set a stage holds the five aligned words around its 8 scales and the two
// zero-point words its 8 rows can touch (lanes 0-13, one word each).
template <int ACT> struct Unit<MOE_W_GPTQ_INT4, ACT> {
    static constexpr int SPAN = 64, CHUNKS = 2, BYTES = 512 + 64;
    static constexpr bool X_RING = false, X_PERM = true, GROUPED = true, ROW_SCALE = false;
    struct Src {
        const uint8_t* p;   // row a + g, k piece c
        const uint8_t* pg;  // the lane's scale or zero-point word, group 0
        int db;             // bytes from row set a to row set b
        int N, G, gstep;    // gstep: bytes from group to group
        bool va, vb, vg;
        __device__ __forceinline__ void aim(const WBase& b, const UnitRows& u, int lane) {
            const int g = lane >> 2, c = lane & 3;
            N = b.N;
            G = b.G;
            va = g < u.na;
            vb = g < u.nb;
            p = b.w + (static_cast<size_t>(c) * N + u.a + g) * 4;
            db = (u.b - u.a) * 4;
            if (lane < 10) {
                const int set = lane / 5, n = ((set ? u.b : u.a) & ~1) + 2 * (lane - 5 * set);
                vg = n < N;
                pg = b.sc + static_cast<size_t>(n) * 2;
                gstep = 2 * N;
            } else {
                const int set = ((lane - 10) >> 1) & 1, n8 = (set ? u.b : u.a) / 8 + (lane & 1);
                vg = lane < 14 && n8 < N / 8;
                pg = b.z + static_cast<size_t>(n8) * 4;
                gstep = N / 2;
            }
        }
        __device__ __forceinline__ void load(uint8_t* st, int k0, int K, bool, int lane) const {
            const uint8_t* w = p + (k0 >> 1) * N;  // k0 / 8 words of 4 bytes
            const int half = 16 * N;
            if (va) {
                cp_async4(st + 4 * lane, w);
                cp_async4(st + 128 + 4 * lane, w + half);
            }
            if (vb) {
                cp_async4(st + 256 + 4 * lane, w + db);
                cp_async4(st + 384 + 4 * lane, w + db + half);
            }
            if (vg) cp_async4(st + 512 + 4 * lane, pg + static_cast<size_t>(k0 / G) * gstep);
        }
    };
    uint32_t w[2][2];  // [row][piece]
    uint32_t z[2];
    float s[2];
    __device__ __forceinline__ void open(const uint8_t* st, const UnitRows& u, int lane) {
        const int g = lane >> 2;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int n = (q ? u.b : u.a), r = n + g;
            w[q][0] = *reinterpret_cast<const uint32_t*>(st + 256 * q + 4 * lane);
            w[q][1] = *reinterpret_cast<const uint32_t*>(st + 256 * q + 128 + 4 * lane);
            s[q] = __half2float(*reinterpret_cast<const __half*>(st + 512 + 20 * q + 2 * ((n & 1) + g)));
            const uint32_t zw = *reinterpret_cast<const uint32_t*>(st + 512 + 40 + 8 * q + 4 * (r / 8 - n / 8));
            z[q] = (zw >> (4 * (r & 7))) & 15u;
        }
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 8 * (c + 4 * i); }
    __device__ __forceinline__ void row(int q, int i, uint32_t (&o)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (k_j, k_{j+4})
            if (ACT == MOE_ACT_F16) {
                const uint32_t v = gemm::and_or(w[q][i] >> (4 * j), 0x000F000Fu, 0x64006400u);  // 1024 + q
                const __half2 zz = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6400u | z[q])));
                const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), zz);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            } else {
                const uint32_t v = gemm::and_or(w[q][i] >> (4 * j), 0x000F000Fu, 0x43004300u);  // 128 + q
                const __nv_bfloat162 zz =
                    __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(0x4300u | z[q])));
                const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), zz);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            }
        }
    }
    __device__ __forceinline__ void frag(int i, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        row(0, i, a);
        row(1, i, b);
    }
    __device__ __forceinline__ float row_scale(int q) const { return s[q]; }
};

// A stage of a warp's ring
template <class U> struct Stage {
    static constexpr int X_AT = U::BYTES, BYTES = (U::BYTES + (U::X_RING ? 512 * U::CHUNKS : 0) + 15) / 16 * 16;
};

__device__ __forceinline__ uint4 perm_0415(const uint4& x) {
    return make_uint4(gemm::prmt(x.x, x.z, 0x5410), gemm::prmt(x.x, x.z, 0x7632), gemm::prmt(x.y, x.w, 0x5410),
                      gemm::prmt(x.y, x.w, 0x7632));
}

// The first token tile's values of one unit. x: the lane's token row (token g),
// already at its piece 0 of contraction index 0, or NULL (no token: zeros).
template <class U> struct Tokens {
    uint4 v[U::CHUNKS];
    // into the stage (X_RING)
    static __device__ __forceinline__ void copy(uint8_t* st, const uint16_t* x, int k0, int K, bool tail, int lane) {
        if (!x) return;
#pragma unroll
        for (int i = 0; i < U::CHUNKS; ++i) {
            const int o = U::k_of(i, 0);
            const bool in = !tail || k0 + U::k_of(i, lane & 3) < K;
            cp_async16_l1(st + 512 * i + 16 * lane, x + (in ? k0 + o : 0), in);
        }
    }
    __device__ __forceinline__ void open(const uint8_t* st, const uint16_t* x, int lane) {
#pragma unroll
        for (int i = 0; i < U::CHUNKS; ++i)
            v[i] = x ? *reinterpret_cast<const uint4*>(st + 512 * i + 16 * lane) : make_uint4(0u, 0u, 0u, 0u);
    }
    // straight into registers
    __device__ __forceinline__ void fetch(const uint16_t* x, int k0, int K, bool tail, int lane) {
#pragma unroll
        for (int i = 0; i < U::CHUNKS; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (x && (!tail || k0 + U::k_of(i, lane & 3) < K))
                v[i] = *reinterpret_cast<const uint4*>(x + k0 + U::k_of(i, 0));
        }
    }
};

// acc[tile] += unit x tokens, for nt tiles of 8 tokens; xp[tile], for tile >= 1, as Tokens' x.
template <class U, int ACT, int NT>
__device__ __forceinline__ void unit_mma(const U& u, const Tokens<U>& x0, const uint16_t* const (&xp)[NT], int nt,
                                         int k0, int K, bool tail, int lane, float (&acc)[NT][4]) {
    float part[NT][4];
    if (U::GROUPED) {
#pragma unroll
        for (int t = 0; t < NT; ++t) part[t][0] = part[t][1] = part[t][2] = part[t][3] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < U::CHUNKS; ++i) {
        uint32_t a[4], b[4];
        u.frag(i, a, b);
        {
            const uint4 x = U::X_PERM ? perm_0415(x0.v[i]) : x0.v[i];
            float (&d)[4] = U::GROUPED ? part[0] : acc[0];
            mma_16816<ACT>(d, a[0], b[0], a[1], b[1], x.x, x.y);
            mma_16816<ACT>(d, a[2], b[2], a[3], b[3], x.z, x.w);
        }
        if (NT > 1 && nt > 1) {
#pragma unroll
            for (int t = 1; t < NT; ++t) {
                if (t >= nt) break;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (xp[t] && (!tail || k0 + U::k_of(i, lane & 3) < K))
                    x = *reinterpret_cast<const uint4*>(xp[t] + k0 + U::k_of(i, 0));
                if (U::X_PERM) x = perm_0415(x);
                float (&d)[4] = U::GROUPED ? part[t] : acc[t];
                mma_16816<ACT>(d, a[0], b[0], a[1], b[1], x.x, x.y);
                mma_16816<ACT>(d, a[2], b[2], a[3], b[3], x.z, x.w);
            }
        }
    }
    if (U::GROUPED) {
        const float s0 = u.row_scale(0), s1 = u.row_scale(1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t > 0 && t >= nt) break;
            acc[t][0] = fmaf(s0, part[t][0], acc[t][0]);
            acc[t][1] = fmaf(s0, part[t][1], acc[t][1]);
            acc[t][2] = fmaf(s1, part[t][2], acc[t][2]);
            acc[t][3] = fmaf(s1, part[t][3], acc[t][3]);
        }
    }
}

}  // namespace moe
