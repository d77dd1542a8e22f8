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
// A "unit" is what a warp takes at a time: two or four 16-row tiles x SPAN
// contraction indices, 2 KB of weights. Units arrive by cp.async in a
// ring of shared-memory stages private to the warp. Each lane copies what it
// will itself read (only scales cross lanes), so a stage needs no barrier
// beyond the warp's own, and what is in flight takes no registers. (The same
// ring in registers ran at a fifth of HBM's rate: loads and conversions kept
// the ring's registers from staying in flight.)
#pragma once

#include "gemm_dequant.cuh"
#include "quant.cuh"

namespace moe {

__device__ __forceinline__ void cp_async4_zfill(void* dst, const void* src, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(full ? 4 : 0)
                 : "memory");
}
// 16 bytes of a weight row, which is read on from there: L2 fetches the 256 bytes around them
__device__ __forceinline__ void cp_async16_row(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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

// Unit<FMT, ACT, GU>: one format's stage layout and fragments, for the gate/up
// kernel (GU: set a holds gate rows, set b the up rows of the same columns) or
// the down kernel (set b holds the rows 8 below those of set a).
//   MT         16-row tiles per unit; SPAN contraction indices; CHUNKS pieces
//              of 8 contraction indices a lane holds per row
//   ROWS       rows of a unit, of each set (GU) or in all (down)
//   ALIGN      first rows are multiples of it
//   row_a / row_b   which rows lane group g has in tile m (row_b: down only)
//   BYTES      weights and scales of a unit in a stage
//   X_RING     the first token tile's values ride in the stage too (formats
//              whose conversion is too short to hide their latency)
//   X_PERM     the token operand's 8 values go in the order 0,4,1,5,2,6,3,7
//   GROUPED    sums of 64 contraction indices are scaled (scale) before they
//              are added to the others
//   SCALE_UP   the sums come out divided by it
//   Src        where a lane copies from: aim() sets it to an expert's rows at
//              a contraction index, load() copies a unit, step() moves on
//   open       reads a stage's words and scales into registers
//   frag(i, m) piece i of both sets of tile m as A operands of two products
// Copies past the contraction's end are filled with zeros (the token operand
// too); a row past the unit's rows is not copied: it only feeds sums that
// nobody reads.
template <int FMT, int ACT, bool GU> struct Unit;

// Rows of K contiguous elements of EB bits, 16 bytes of each row and lane;
// tiles DOWN rows apart.
template <int EB, int MT, int DOWN> struct RowSrc {
    const uint8_t* pa;
    const uint8_t* pb;
    int na, nb, tile;  // tiles in which the lane's rows exist; bytes from tile to tile
    __device__ __forceinline__ void aim(const WBase& b, int a, int n_a, int bb, int n_b, int k0, int lane) {
        const int g = lane >> 2, k = k0 + (lane & 3) * (128 / EB);
        na = (n_a - g + DOWN - 1) / DOWN;
        nb = (n_b - g + DOWN - 1) / DOWN;
        tile = b.K * EB / 8 * DOWN;
        pa = b.w + (static_cast<size_t>(a + g) * b.K + k) * EB / 8;
        pb = b.w + (static_cast<size_t>(bb + g) * b.K + k) * EB / 8;
    }
    __device__ __forceinline__ void load(uint8_t* st, int lane) const {
        uint8_t* d = st + 16 * lane;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m < na) cp_async16_row(d + 1024 * m, pa + m * tile);
            if (m < nb) cp_async16_row(d + 1024 * m + 512, pb + m * tile);
        }
    }
    __device__ __forceinline__ void load_tail(uint8_t* st, int left, int lane) const {  // `left` indices to K's end
        uint8_t* d = st + 16 * lane;
        const bool in = (lane & 3) * (128 / EB) < left;
        const int o = in ? 0 : -16 * (lane & 3);  // a skipped copy reads nothing: the unit's first piece stands in
        for (int m = 0; m < MT; ++m) {
            if (m < na) cp_async16_zfill(d + 1024 * m, pa + m * tile + o, in);
            if (m < nb) cp_async16_zfill(d + 1024 * m + 512, pb + m * tile + o, in);
        }
    }
    __device__ __forceinline__ void step() {
        pa += 64;
        pb += 64;
    }
};

template <int ACT, bool GU> struct Unit<MOE_W_BF16, ACT, GU> {
    static constexpr int MT = 2, SPAN = 32, CHUNKS = 1, BYTES = 1024 * MT;
    static constexpr int DOWN = GU ? 8 : 16, ROWS = DOWN * MT, ALIGN = 1;
    static constexpr bool X_RING = true, X_PERM = false, GROUPED = false, ROW_SCALE = false;
    static constexpr float SCALE_UP = 1.0f;
    struct Src : RowSrc<16, MT, DOWN> {};
    uint4 r[MT][2];
    static __device__ __forceinline__ int row_a(int m, int g) { return DOWN * m + g; }
    static __device__ __forceinline__ int row_b(int m, int g) { return DOWN * m + 8 + g; }
    __device__ __forceinline__ void open(const uint8_t* st, int, int, int lane) {
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) r[q / 2][q % 2] = *reinterpret_cast<const uint4*>(st + 512 * q + 16 * lane);
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 8 * c + 32 * i; }
    __device__ __forceinline__ void frag(int, int m, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        a[0] = r[m][0].x; a[1] = r[m][0].y; a[2] = r[m][0].z; a[3] = r[m][0].w;
        b[0] = r[m][1].x; b[1] = r[m][1].y; b[2] = r[m][1].z; b[3] = r[m][1].w;
    }
    __device__ __forceinline__ float scale(int, int, int) const { return 1.0f; }
};

template <int ACT, bool GU> struct Unit<MOE_W_FP8_E4M3, ACT, GU> {
    static constexpr int MT = 2, SPAN = 64, CHUNKS = 2, BYTES = 1024 * MT;
    static constexpr int DOWN = GU ? 8 : 16, ROWS = DOWN * MT, ALIGN = 1;
    static constexpr bool X_RING = false, X_PERM = false, GROUPED = false, ROW_SCALE = true;
    static constexpr float SCALE_UP = 1.0f;
    struct Src : RowSrc<8, MT, DOWN> {};
    uint4 r[MT][2];
    static __device__ __forceinline__ int row_a(int m, int g) { return DOWN * m + g; }
    static __device__ __forceinline__ int row_b(int m, int g) { return DOWN * m + 8 + g; }
    __device__ __forceinline__ void open(const uint8_t* st, int, int, int lane) {
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) r[q / 2][q % 2] = *reinterpret_cast<const uint4*>(st + 512 * q + 16 * lane);
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 16 * c + 8 * i; }
    __device__ __forceinline__ void frag(int i, int m, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        const uint4 &u = r[m][0], &v = r[m][1];
        e4m3x4_to_act<ACT>(i & 1 ? u.z : u.x, a[0], a[1]);
        e4m3x4_to_act<ACT>(i & 1 ? u.w : u.y, a[2], a[3]);
        e4m3x4_to_act<ACT>(i & 1 ? v.z : v.x, b[0], b[1]);
        e4m3x4_to_act<ACT>(i & 1 ? v.w : v.y, b[2], b[3]);
    }
    __device__ __forceinline__ float scale(int, int, int) const { return 1.0f; }
};

// NVFP4: the block scales lie along n, one byte each. For each of the unit's 8
// blocks a stage holds the aligned words around the unit's rows: WS words for
// each of SETS runs of rows (gate and up), three words a lane at most.
//
// To bf16, a pair of codes takes two shifts and two logic operations: sign to
// bit 15, exponent and mantissa to bits 8..6, which is the code's value times
// 2^-126 (subnormals included). The block scale carries 2^118 of that back
// (448 * 2^118 is the most that fits) and the finished sums the other 2^8; the
// product is exact, as 6 significant bits are.
template <int ACT, bool GU> struct Unit<MOE_W_NVFP4, ACT, GU> {
    static constexpr int MT = 2, SPAN = 128, CHUNKS = 4;
    static constexpr int DOWN = GU ? 8 : 16, ROWS = DOWN * MT, ALIGN = 1;
    static constexpr int SETS = GU ? 2 : 1, WS = ROWS / 4 + 1;  // words around ROWS unaligned bytes
    static constexpr int WORDS = 8 * SETS * WS, SC_AT = 1024 * MT, BYTES = SC_AT + WORDS * 4;
    static constexpr bool X_RING = false, X_PERM = ACT == MOE_ACT_BF16, GROUPED = false, ROW_SCALE = false;
    static constexpr float SCALE_UP = ACT == MOE_ACT_BF16 ? 256.0f : 1.0f;
    static constexpr int PIECES = (WORDS + 31) / 32;
    struct Src : RowSrc<4, MT, DOWN> {
        const uint8_t* ps[PIECES];
        uint32_t ok;  // bit h: piece h exists
        int row_step;
        __device__ __forceinline__ void aim(const WBase& b, int a, int n_a, int bb, int n_b, int k0, int lane) {
            RowSrc<4, MT, DOWN>::aim(b, a, n_a, bb, n_b, k0, lane);
            row_step = 8 * b.N;
            ok = 0;
#pragma unroll
            for (int h = 0; h < PIECES; ++h) {
                const int p = lane + 32 * h, set = p / (8 * WS), q = p - 8 * WS * set;
                const int n = ((set ? bb : a) & ~3) + 4 * (q % WS);
                if (p < WORDS && n < b.N) ok |= 1u << h;
                ps[h] = b.sc + static_cast<size_t>(k0 / 16 + q / WS) * b.N + n;
            }
        }
        __device__ __forceinline__ void load(uint8_t* st, int lane) const {
            RowSrc<4, MT, DOWN>::load(st, lane);
#pragma unroll
            for (int h = 0; h < PIECES; ++h)
                if (ok >> h & 1) cp_async4(st + SC_AT + 128 * h + 4 * lane, ps[h]);
        }
        __device__ __forceinline__ void load_tail(uint8_t* st, int left, int lane) const {
            RowSrc<4, MT, DOWN>::load_tail(st, left, lane);
            for (int h = 0; h < PIECES; ++h) {
                // a scale past the end meets zero codes, but must not be a NaN
                const int kb = (lane + 32 * h) % (8 * WS) / WS;
                const bool in = 16 * kb < left;
                if (ok >> h & 1)
                    cp_async4_zfill(st + SC_AT + 128 * h + 4 * lane, in ? ps[h] : ps[h] - kb * (row_step / 8), in);
            }
        }
        __device__ __forceinline__ void step() {
            RowSrc<4, MT, DOWN>::step();
#pragma unroll
            for (int h = 0; h < PIECES; ++h) ps[h] += row_step;
        }
    };
    uint4 r[MT][2];
    uint32_t s2[MT][2][2];  // the two block scales of the lane's 32 codes, each twice in a word
    static __device__ __forceinline__ int row_a(int m, int g) { return DOWN * m + g; }
    static __device__ __forceinline__ int row_b(int m, int g) { return DOWN * m + 8 + g; }
    __device__ __forceinline__ void open(const uint8_t* st, int a, int b, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                r[m][h] = *reinterpret_cast<const uint4*>(st + 512 * (2 * m + h) + 16 * lane);
                const uint8_t* s = GU ? st + SC_AT + (h * 8 + 2 * c) * WS * 4 + ((h ? b : a) & 3) + 8 * m + g
                                      : st + SC_AT + 2 * c * WS * 4 + (a & 3) + 16 * m + 8 * h + g;
                uint32_t f;
                asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
                    : "=r"(f)
                    : "r"(s[0] | (static_cast<uint32_t>(s[WS * 4]) << 8)));
                if (ACT == MOE_ACT_F16) {
                    s2[m][h][0] = gemm::prmt(f, f, 0x1010u);
                    s2[m][h][1] = gemm::prmt(f, f, 0x3232u);
                } else {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
                    const float lo = v.x * 0x1p118f, hi = v.y * 0x1p118f;
                    s2[m][h][0] = Act<MOE_ACT_BF16>::pack2(lo, lo);
                    s2[m][h][1] = Act<MOE_ACT_BF16>::pack2(hi, hi);
                }
            }
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 32 * c + 8 * i; }
    static __device__ __forceinline__ void row(const uint4& w, uint32_t m, int i, uint32_t (&o)[4]) {
        const uint32_t word = i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
        if (ACT == MOE_ACT_BF16) {
            // (k_j, k_{j+4})
            o[0] = gemm::and_or(word << 6, 0x01C001C0u, (word << 12) & 0x80008000u);
            o[1] = gemm::and_or(word << 2, 0x01C001C0u, (word << 8) & 0x80008000u);
            o[2] = gemm::and_or(word >> 2, 0x01C001C0u, (word << 4) & 0x80008000u);
            o[3] = gemm::and_or(word >> 6, 0x01C001C0u, word & 0x80008000u);
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
    __device__ __forceinline__ void frag(int i, int m, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        row(r[m][0], s2[m][0][i >> 1], i, a);
        row(r[m][1], s2[m][1][i >> 1], i, b);
    }
    __device__ __forceinline__ float scale(int, int, int) const { return 1.0f; }
};

// GPTQ: the words of 8 k values lie along n, so a lane copies four neighbouring
// columns' words at once and they go to four different rows of its fragments:
//   gate/up  lane group g has columns 4g .. 4g + 3, one in each of four tiles
//            (32 columns an item, a 128-byte line per k word; with 8 columns an
//            item, DRAM read 3.3 times the weights)
//   down     columns 4g .. 4g + 3 are rows g and g + 8 of two tiles
// The fragments hold the integers q - z (exact), and the group's f16 scale
// multiplies the f32 sums of each 64 contraction indices (a divisor of every
// group). Per 64 indices a lane group's four scales and its zero-point word are
// copied by one lane each: lane c = 0 / 1 scales of set a / b, 2 / 3 zeros.
template <int ACT, bool GU> struct Unit<MOE_W_GPTQ_INT4, ACT, GU> {
    static constexpr int V = 4, SETS = GU ? 2 : 1, KT = GU ? 1 : 2;  // KT: pieces of 64 indices
    static constexpr int MT = GU ? 4 : 2, SPAN = 64 * KT, CHUNKS = 2 * KT;
    static constexpr int ROWS = 32, ALIGN = V;
    static constexpr int PIECE = 32 * 4 * V;                    // bytes of one k word of all lanes
    static constexpr int SC_AT = 2 * KT * SETS * PIECE;         // then, per 64 indices and set: scales, zeros
    static constexpr int SC_SET = 8 * (2 * V + 4), BYTES = SC_AT + KT * SETS * SC_SET;
    static constexpr bool X_RING = false, X_PERM = true, GROUPED = true, ROW_SCALE = false;
    static constexpr float SCALE_UP = 1.0f;
    struct Src {
        const uint8_t* p;   // set a, k word c
        const uint8_t* pg;  // the lane's scales or zero-point word of the group
        int N, db, gstep;   // gstep: bytes from group to group
        int per, rest;      // 64s of contraction indices in a group, and left of this one
        bool va, vb, vg;
        __device__ __forceinline__ void aim(const WBase& b, int a, int n_a, int bb, int n_b, int k0, int lane) {
            const int g = lane >> 2, c = lane & 3, set = GU ? c & 1 : 0, n = (set ? bb : a) + V * g;
            N = b.N;
            per = b.G / 64;
            const int group = k0 / b.G;
            rest = per - (k0 - group * b.G) / 64;
            va = V * g < n_a;
            vb = V * g < n_b;
            db = (bb - a) * 4;
            p = b.w + (static_cast<size_t>(k0 / 8 + c) * N + a + V * g) * 4;
            vg = (set ? vb : va) && (GU || c == 0 || c == 2);
            if (c < 2) {
                pg = b.sc + static_cast<size_t>(n) * 2;
                gstep = 2 * N;
            } else {
                pg = b.z + static_cast<size_t>(n / 8) * 4;
                gstep = N / 2;
            }
            pg += static_cast<size_t>(group) * gstep;
        }
        __device__ __forceinline__ void load_n(uint8_t* st, int left, int lane) {
            uint8_t* d = st + 4 * V * lane;
            const int half = 16 * N;  // 4 k words on
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const bool in = 64 * t < left;
                const uint8_t* w = in ? p + 2 * t * half : p;
                if (va) {
                    cp_async16_zfill(d + 2 * t * PIECE, w, in);
                    cp_async16_zfill(d + (2 * t + 1) * PIECE, w + half, in);
                }
                if (GU && vb) {
                    cp_async16_zfill(d + 2 * PIECE, w + db, in);
                    cp_async16_zfill(d + 3 * PIECE, w + db + half, in);
                }
                if (vg) {
                    const int g = lane >> 2, c = lane & 3;
                    uint8_t* s = st + SC_AT + (t * SETS + (GU ? c & 1 : 0)) * SC_SET;
                    if (c >= 2)
                        cp_async4_zfill(s + 16 * V + 4 * g, pg, in);
                    else
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(s + 8 * g)), "l"(pg),
                                     "r"(in ? 8 : 0)
                                     : "memory");
                }
                // on by 64 indices; not past the end, where the last group stands in for a copy of nothing
                if (--rest == 0) {
                    rest = per;
                    if (64 * (t + 1) < left) pg += gstep;
                }
            }
        }
        __device__ __forceinline__ void load(uint8_t* st, int lane) { load_n(st, 1 << 30, lane); }
        __device__ __forceinline__ void load_tail(uint8_t* st, int left, int lane) { load_n(st, left, lane); }
        __device__ __forceinline__ void step() { p += static_cast<size_t>(KT) * 32 * N; }
    };
    uint32_t w[KT][2][SETS][V];
    uint32_t z[KT][SETS];  // the V zero points, 4 bits each
    uint2 s[KT][SETS];     // the V scales
    static __device__ __forceinline__ int row_a(int m, int g) { return GU ? 4 * g + m : 4 * g + 2 * m; }
    static __device__ __forceinline__ int row_b(int m, int g) { return 4 * g + 2 * m + 1; }
    __device__ __forceinline__ void open(const uint8_t* st, int a, int b, int lane) {
        const int g = lane >> 2;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int q = 0; q < SETS; ++q) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 u = *reinterpret_cast<const uint4*>(st + (2 * (t * SETS + q) + i) * PIECE + 16 * lane);
                    w[t][i][q][0] = u.x;
                    w[t][i][q][1] = u.y;
                    w[t][i][q][2] = u.z;
                    w[t][i][q][3] = u.w;
                }
                const uint8_t* sc = st + SC_AT + (t * SETS + q) * SC_SET;
                s[t][q] = *reinterpret_cast<const uint2*>(sc + 8 * g);
                z[t][q] = *reinterpret_cast<const uint32_t*>(sc + 16 * V + 4 * g) >> (4 * (((q ? b : a) + V * g) & 7));
            }
    }
    static __device__ __forceinline__ int k_of(int i, int c) { return 8 * c + 32 * i; }
    static __device__ __forceinline__ void row(uint32_t w, uint32_t z, uint32_t (&o)[4]) {  // (k_j, k_{j+4})
        if (ACT == MOE_ACT_F16) {
            // 1024 + q, or 1024 + 16 q (divided by 16 again); both differences are exact
            const __half2 z1 = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6400u | z)));
            const __half2 nz = __half2half2(__ushort_as_half(static_cast<unsigned short>(0xD400u | (z << 4))));  // -(64 + z)
            const __half2 c16 = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x2C00u)));
            const uint32_t w8 = w >> 8;
            const uint32_t q[4] = {gemm::and_or(w, 0x000F000Fu, 0x64006400u), gemm::and_or(w, 0x00F000F0u, 0x64006400u),
                                   gemm::and_or(w8, 0x000F000Fu, 0x64006400u),
                                   gemm::and_or(w8, 0x00F000F0u, 0x64006400u)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = *reinterpret_cast<const __half2*>(&q[j]);
                const __half2 d = (j & 1) ? __hfma2(h, c16, nz) : __hsub2(h, z1);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            }
        } else {
            const __nv_bfloat162 zz = __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(0x4300u | z)));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t v = gemm::and_or(w >> (4 * j), 0x000F000Fu, 0x43004300u);  // 128 + q
                const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), zz);
                o[j] = *reinterpret_cast<const uint32_t*>(&d);
            }
        }
    }
    __device__ __forceinline__ void frag(int i, int m, uint32_t (&a)[4], uint32_t (&b)[4]) const {
        const int t = i >> 1;
        if (GU) {
            row(w[t][i & 1][0][m], (z[t][0] >> (4 * m)) & 15u, a);
            row(w[t][i & 1][SETS - 1][m], (z[t][SETS - 1] >> (4 * m)) & 15u, b);
        } else {
            row(w[t][i & 1][0][(2 * m) & 3], (z[t][0] >> (8 * m)) & 15u, a);
            row(w[t][i & 1][0][(2 * m + 1) & 3], (z[t][0] >> (8 * m + 4)) & 15u, b);
        }
    }
    // of piece i's group: row a (h = 0) or b of tile m
    __device__ __forceinline__ float scale(int i, int m, int h) const {
        const int t = i >> 1, v = GU ? m : 2 * m + h;
        const uint2& u = s[t][GU ? h * (SETS - 1) : 0];
        const uint32_t word = v < 2 ? u.x : u.y;
        return __half2float(__ushort_as_half(static_cast<unsigned short>(v & 1 ? word >> 16 : word & 0xffffu)));
    }
};

// A stage of a warp's ring
template <class U> struct Stage {
    static constexpr int X_AT = (U::BYTES + 15) / 16 * 16, BYTES = X_AT + (U::X_RING ? 512 * U::CHUNKS : 0);
};

__device__ __forceinline__ uint4 perm_0415(const uint4& x) {
    return make_uint4(gemm::prmt(x.x, x.z, 0x5410), gemm::prmt(x.x, x.z, 0x7632), gemm::prmt(x.y, x.w, 0x5410),
                      gemm::prmt(x.y, x.w, 0x7632));
}
// 16 bytes where `ok`, else v as it was
__device__ __forceinline__ void ld16_if(uint4& v, const void* p, bool ok) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"(static_cast<int>(ok))
        : "memory");
}

// The first token tile's values of one unit. x: the lane's token row (token g)
// at the unit's first contraction index, already moved to the lane's piece 0;
// `has`: whether there is such a token (else zeros).
template <class U> struct Tokens {
    uint4 v[U::CHUNKS];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < U::CHUNKS; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // into the stage (X_RING); `left`: contraction indices to the end, SPAN or more if none are missing
    static __device__ __forceinline__ void copy(uint8_t* st, const uint16_t* x, bool has, int left, int lane) {
        if (!has) return;
#pragma unroll
        for (int i = 0; i < U::CHUNKS; ++i) {
            const bool in = U::k_of(i, lane & 3) < left;
            cp_async16_l1(st + 512 * i + 16 * lane, x + (in ? U::k_of(i, 0) : -U::k_of(0, lane & 3)), in);
        }
    }
    // from the stage; lanes without a token keep what clear() left
    __device__ __forceinline__ void open(const uint8_t* st, bool has, int lane) {
        if (has)
#pragma unroll
            for (int i = 0; i < U::CHUNKS; ++i) v[i] = *reinterpret_cast<const uint4*>(st + 512 * i + 16 * lane);
    }
    // straight into registers
    __device__ __forceinline__ void fetch(const uint16_t* x, bool has, int left, int lane) {
        if (left >= U::SPAN) {
#pragma unroll
            for (int i = 0; i < U::CHUNKS; ++i) ld16_if(v[i], x + U::k_of(i, 0), has);
        } else {
            clear();
#pragma unroll
            for (int i = 0; i < U::CHUNKS; ++i) ld16_if(v[i], x + U::k_of(i, 0), has && U::k_of(i, lane & 3) < left);
        }
    }
};

// acc[tile][token tile] += unit x tokens, for the first NT of NTA token tiles of
// 8. x1, has1: the lane's token of the second tile, as in Tokens.
template <class U, int ACT, int NT, int NTA>
__device__ __forceinline__ void unit_mma_n(const U& u, const Tokens<U>& x0, const uint16_t* x1, bool has1, int left,
                                           int lane, float (&acc)[U::MT][NTA][4]) {
    float part[U::MT][NT][4];
#pragma unroll
    for (int i = 0; i < U::CHUNKS; ++i) {
        if (U::GROUPED && (i & 1) == 0) {
#pragma unroll
            for (int m = 0; m < U::MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) part[m][t][0] = part[m][t][1] = part[m][t][2] = part[m][t][3] = 0.0f;
        }
        uint4 x[NT];
        x[0] = U::X_PERM ? perm_0415(x0.v[i]) : x0.v[i];
        if (NT > 1) {
            x[NT - 1] = make_uint4(0u, 0u, 0u, 0u);
            ld16_if(x[NT - 1], x1 + U::k_of(i, 0), has1 && U::k_of(i, lane & 3) < left);
            if (U::X_PERM) x[NT - 1] = perm_0415(x[NT - 1]);
        }
#pragma unroll
        for (int m = 0; m < U::MT; ++m) {
            uint32_t a[4], b[4];
            u.frag(i, m, a, b);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float (&d)[4] = U::GROUPED ? part[m][t] : acc[m][t];
                mma_16816<ACT>(d, a[0], b[0], a[1], b[1], x[t].x, x[t].y);
                mma_16816<ACT>(d, a[2], b[2], a[3], b[3], x[t].z, x[t].w);
            }
        }
        if (U::GROUPED && (i & 1) == 1) {
#pragma unroll
            for (int m = 0; m < U::MT; ++m) {
                const float s0 = u.scale(i, m, 0), s1 = u.scale(i, m, 1);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[m][t][0] = fmaf(s0, part[m][t][0], acc[m][t][0]);
                    acc[m][t][1] = fmaf(s0, part[m][t][1], acc[m][t][1]);
                    acc[m][t][2] = fmaf(s1, part[m][t][2], acc[m][t][2]);
                    acc[m][t][3] = fmaf(s1, part[m][t][3], acc[m][t][3]);
                }
            }
        }
    }
}
template <class U, int ACT, int NT>
__device__ __forceinline__ void unit_mma(const U& u, const Tokens<U>& x0, const uint16_t* x1, bool has1, int nt,
                                         int left, int lane, float (&acc)[U::MT][NT][4]) {
    if (NT == 1 || nt == 1) unit_mma_n<U, ACT, 1, NT>(u, x0, x1, has1, left, lane, acc);
    else unit_mma_n<U, ACT, NT, NT>(u, x0, x1, has1, left, lane, acc);
}

}  // namespace moe
