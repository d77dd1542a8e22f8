// Products grouped by expert over ragged spans, their gradients, and the dense
// product with its epilogue: entry points.
#include "ragged.cuh"
#include <math.h>

namespace moe {
namespace {

// Which form a product of rows takes.
//
// Groups whose sizes only the device knows: CTA pairs, tiles of up to twice a group's mean
// rows (3066 rows of 64 groups, most of 30 to 60: 71 us with tiles of 96 rows, 72 of 128, 74
// of 256, whose over-wide boxes bring rows of the next groups along, 80 of 48, which read
// the fuller groups' weights more than once); or, of at most 128 rows in all and few tiles,
// the split form, by the same model with as many groups as rows dealt at random touch (34 rows
// of 4 groups, 12320 x 840 transposed: pairs 45 us, split 21; 100 rows of 16 groups, 512 x 512: 7.1 and 5.7).
//
// One group (a dense product): the form, row tiles and split that a model of their time
// finds best. Its costs (ns) were fitted to 110 sizes from 1 x 88 x 88 to 4000 x 2048 x 14336
// at an earlier state of the kernels, whose epilogues have become faster since, and it knows
// nothing of bias, function, residual and z. Against the best of all forms, on 70 random sizes
// that the fit did not see: half of the choices lose 0.1% or less, the mean 6%. It loses most
// at streaming's rows with contractions below 600, for whose tile ends it has no term (14
// sizes: 13% in the mean; 17 x 27104 x 120 12.0 us, split 6.5; 32 x 28672 x 64 15.0 and 4.3), with
// full epilogues (6 sizes: 17%, 37% at worst), and at single sizes (2676 x 1712 x 13448: pairs of
// 16 units 182 us, of 10 130); transposed products lose 1%.
//   streaming (up to 32 rows): the weights at 5.7 TB/s, or a warp's blocks one after the
//     other, and 27 ps a byte of the rows, which every CTA reads
//   split: a launch (and its clusters' meetings), a CTA's blocks, slower where two share an
//     SM, or the weights at 5.6 TB/s; 26 a row of the tile at its end
//   pairs: waves of tiles, each its blocks or its epilogue, or the weights at 5 TB/s
// (us, streaming / split / pairs: 1 x 2816 x 2048 4.8 / 8.2 / 12.8; 32 x 2816 x 2048 9.2 / 8.7 / 13.1; 16 x
// 14336 x 4096 26.6 / 24.7 / 27.8; 64 x 4096 x 14336 - / 27.6 / 52.6; 333 x 2816 x 2048 - / 13.3 / 14.2; 1333 x 2816 x
// 2048 - / 23.1 / 19.6.)
struct RowsPick {
    RowsForm f;
    bool streaming;
};

struct Split {
    int parts, launch_ns;
};
constexpr Split kSplits[] = {{1, 2620}, {2, 4940}, {4, 5410}, {8, 6610}};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

RowsPick pick_rows_form(const RaggedParams& p, bool transposed, int sms) {
    const int64_t U = ceil_div(p.rows, 16), KB = ceil_div(p.C, 64);
    RowsPick best{{1, 0, 0}, false};
    int64_t best_ns = INT64_MAX;
    auto offer = [&](int64_t ns, const RowsPick& pick) {
        if (ns < best_ns) {
            best_ns = ns;
            best = pick;
        }
    };
    const int64_t J = p.J;
    // groups that have rows, and the pairs' row tiles of a group, if all have the same
    int64_t groups = 1, m0 = ceil_div(U, 16), m1 = U < m0 + 7 ? U : m0 + 7;
    if (p.offsets) {
        const int64_t units = ceil_div(ceil_div(p.rows, p.E), 16);
        const int maxu = static_cast<int>(units >= 8 ? 16 : 2 * units);
        if (p.rows > SPLIT_MAX_ROWS) return {{maxu, 0, 0}, false};
        groups = static_cast<int64_t>(ceil(p.E * (1.0 - pow(1.0 - 1.0 / p.E, p.rows))));
        m0 = m1 = 0;
        offer(5130 + max64(ceil_div(groups * ceil_div(J, 256), sms / 2) * max64(KB * 200, 1500),
                           2 * J * p.C * groups / 5000) + 240, {{maxu, 0, 0}, false});
    }
    const int64_t bytes = 2 * J * p.C * groups;
    if (p.rows <= 32 && !transposed && !p.offsets)
        offer(2170 + max64(bytes / 5700, 250 * ceil_div(KB, 8)) + 27 * p.rows * (2 * static_cast<int64_t>(p.C)) / 1024,
              {{0, 0, 0}, true});
    const int64_t mt = p.offsets ? 1 : ceil_div(U, 8), h = p.offsets ? 16 : ceil_div(U, mt) * 16;
    for (const auto& s : kSplits) {
        const int64_t ctas = ceil_div(J, 128) * mt * groups * s.parts;
        if (s.parts > KB || ceil_div(J, 128) * mt * (p.offsets ? p.E : 1) * s.parts > 4 * sms) break;
        const int64_t blocks = ceil_div(KB, s.parts), load = ctas > sms ? 2 : 1;
        const int64_t body = blocks * (198 + h * 11 / 10);
        const int64_t ns = max64(max64(body, load * blocks * (85 + h * 11 / 10)), bytes / 5600) +
                           (ceil_div(ctas, 2 * sms) - 1) * (s.launch_ns + body) + s.launch_ns + 26 * h * load;
        offer(ns, {{0, static_cast<int>(mt), s.parts}, false});
    }
    for (int64_t t = m0; t <= m1 && t > 0; ++t) {
        const int64_t rows = ceil_div(U, t) * 16, waves = ceil_div(t * ceil_div(J, 256), sms / 2);
        const int64_t ns =
            5130 + max64(waves * max64(KB * (189 + rows * 4 / 10), 1300 + 15 * rows), bytes / 5000) + 15 * rows;
        offer(ns, {{static_cast<int>(ceil_div(U, t)), 0, 0}, false});
    }
    return best;
}

// Which form the gradient of a weight takes.
//
// CTA pairs (parts 0): kt tiles of nearly equal width side by side, of 256 columns at most, and
// more of them where they fill the waves of tiles better (12288 rows of 64 groups, 2048 x 1408
// f32 with addends: five of 256 columns and one of 128 278 us, six alike 254, eight 237; 1333
// rows, 2816 x 2048 f32: eight side by side, 88 tiles for 76 pairs, 21.4, thirteen 19.1, both
// before the sums' chunks). A tile takes its blocks of 64 rows, 140 + 0.73 ns a column each,
// and 0.7 us between tiles (2532 rows of 6 groups, 18736 x 944 f32: four side by side 110 us,
// five 122, six 130), or the way of its bytes, 82 a ns, and if they are 16-bit 0.8 us to pack
// them. Over many waves a pair's tiles have the average width.
//
// Of one group with few tiles, the split form: parts CTAs share a tile's rows; its time as
// above, more where two of them share an SM, and for addends, which its lanes read 64 bytes at
// a time. (us, pairs / split, f32: 4000 rows, 512 x 512 20.4 / 12.0; 2000 rows, 2048 x 512 13.5 /
// 12.7; 100 rows, 1000 x 1000 6.2 / 5.5; 30000 rows, 264 x 520 151 / 33; with the forms' models
// the other way, 640 rows, 2048 x 1408 9.4 / 14.0, 100 rows, 1000 x 1000 with addends 7.8 / 10.3.)
struct GradientForm {
    int parts, kt;
};
GradientForm pick_gradient_form(const RaggedParams& p, bool f32, int sms) {
    const int64_t units = ceil_div(p.C, gradient_unit(f32)), widest = 256 / gradient_unit(f32);
    const int64_t kt0 = ceil_div(units, widest);
    GradientForm best{0, static_cast<int>(kt0)};
    if (p.rows == 0 || sms < 2) return best;  // (without a device the launch reports it)
    const int64_t KB = ceil_div(ceil_div(p.rows, p.E), 64), rows = ceil_div(p.J, 256) * p.E;
    const int64_t bytes = f32 ? (p.addend ? 8 : 4) : 2, fixed = f32 ? 0 : 800;
    int64_t best_ns = INT64_MAX;
    for (int64_t kt = kt0; kt <= 2 * kt0 && kt <= kt0 + 12 && kt <= units; ++kt) {
        const int64_t waves = ceil_div(rows * kt, sms / 2);
        const int64_t width = waves > 3 ? p.C / kt : ceil_div(units, kt) * gradient_unit(f32);
        const int64_t ns = 5100 + waves * max64(KB * (140 + width * 73 / 100) + 700, fixed + bytes * 256 * width / 82);
        if (ns < best_ns) {
            best_ns = ns;
            best.kt = static_cast<int>(kt);
        }
    }
    if (p.offsets) return best;
    const int64_t tiles = ceil_div(p.J, 128) * ceil_div(p.C, 128);
    for (const auto& s : kSplits) {
        if (s.parts > KB || tiles * s.parts > 2 * sms) break;
        const int64_t blocks = ceil_div(KB, s.parts);
        const int64_t ns = s.launch_ns + (tiles * s.parts > sms ? 2000 + blocks * 720 : blocks * 230) +
                           (s.parts < 8 ? 2500 : 4000) + (p.addend ? 400 + 4600 / s.parts : 0);
        if (ns < best_ns) {
            best_ns = ns;
            best.parts = s.parts;
        }
    }
    return best;
}

int launch_rows(const RaggedArgs& g) {
    const int sms = sm_count();
    if (sms < 2) return fail(MOE_ERR_CUDA, "%s: no CUDA device", g.who);
    const RowsPick pick = pick_rows_form(g.p, g.transposed, sms);
    if (pick.streaming) return launch_dense_rows(g);
    return g.act == MOE_ACT_BF16 ? launch_ragged_rows_bf16(g, pick.f) : launch_ragged_rows_f16(g, pick.f);
}

int check_shapes(const char* who, int act, const int32_t* offsets, int rows, int N, int K, int E) {
    MOE_REQUIRE(act == MOE_ACT_BF16 || act == MOE_ACT_F16, "%s: act=%d is neither bf16 nor fp16", who, act);
    MOE_REQUIRE(rows >= 0, "%s: %d rows", who, rows);
    MOE_REQUIRE(N > 0 && N % 8 == 0, "%s: N=%d must be a positive multiple of 8", who, N);
    MOE_REQUIRE(K > 0 && K % 8 == 0, "%s: K=%d must be a positive multiple of 8", who, K);
    MOE_REQUIRE(E >= 1 && E <= MOE_MAX_EXPERTS, "%s: E=%d outside [1, %d]", who, E, MOE_MAX_EXPERTS);
    if (rows > (1 << 30) || N > (1 << 30) || K > (1 << 30))
        return fail(MOE_ERR_UNSUPPORTED, "%s: %d rows, N=%d or K=%d above 2^30", who, rows, N, K);
    MOE_REQUIRE(offsets || E == 1, "%s: no offsets, but E=%d groups", who, E);
    MOE_REQUIRE((reinterpret_cast<uintptr_t>(offsets) & 3u) == 0, "%s: offsets must be 4-byte aligned", who);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_ragged_gemm(const void* a, int32_t act, const void* w, int32_t transposed, const int32_t* offsets,
                               int32_t rows, int32_t N, int32_t K, int32_t E, void* out, int32_t* err_word,
                               void* stream) {
    const char* who = "moe_ragged_gemm";
    const int rc = moe::check_shapes(who, act, offsets, rows, N, K, E);
    if (rc != MOE_OK) return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(a && w && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(out), "%s: a / w / out must be 16-byte aligned",
                who);
    moe::RaggedArgs g{};
    g.p.offsets = offsets;
    g.p.rows = rows;
    g.p.E = E;
    g.p.J = transposed ? K : N;
    g.p.C = transposed ? N : K;
    g.p.out = out;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = a;
    g.w = w;
    g.act = act;
    g.transposed = transposed;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    return moe::launch_rows(g);
}

extern "C" int moe_ragged_wgrad(const void* dy, const void* x, int32_t act, const int32_t* offsets, int32_t rows,
                                int32_t N, int32_t K, int32_t E, const float* addend, void* dw, int32_t dw_f32,
                                int32_t* err_word, void* stream) {
    const char* who = "moe_ragged_wgrad";
    const int rc = moe::check_shapes(who, act, offsets, rows, N, K, E);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(dw_f32 || !addend, "%s: an addend goes with an f32 gradient", who);
    MOE_REQUIRE(dw && (rows == 0 || (dy && x)), "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(dy) && moe::aligned16(x) && moe::aligned16(addend) && moe::aligned16(dw),
                "%s: tensors must be 16-byte aligned", who);
    moe::RaggedArgs g{};
    g.p.offsets = offsets;
    g.p.rows = rows;
    g.p.E = E;
    g.p.J = N;
    g.p.C = K;
    g.p.out = dw;
    g.p.addend = addend;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = dy;
    g.w = x;
    g.act = act;
    g.f32 = dw_f32;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    const moe::GradientForm form = moe::pick_gradient_form(g.p, dw_f32 != 0, moe::sm_count());
    g.parts = form.parts;
    g.kt = form.kt;
    return moe::launch_ragged_wgrad(g);
}

extern "C" int moe_dense_gemm(const void* a, int32_t act, const void* w, const void* bias, int32_t fn,
                              const void* residual, void* pre, void* out, int32_t M, int32_t N, int32_t K,
                              int32_t* err_word, void* stream) {
    const char* who = "moe_dense_gemm";
    const int rc = moe::check_shapes(who, act, nullptr, M, N, K, 1);
    if (rc != MOE_OK) return rc;
    MOE_REQUIRE(fn >= MOE_FN_NONE && fn <= MOE_FN_SILU, "%s: unknown activation function %d", who, fn);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(a && w && out, "%s: NULL pointer", who);
    MOE_REQUIRE(moe::aligned16(a) && moe::aligned16(w) && moe::aligned16(bias) && moe::aligned16(residual) &&
                    moe::aligned16(pre) && moe::aligned16(out),
                "%s: tensors must be 16-byte aligned", who);
    moe::RaggedArgs g{};
    g.p.rows = M;
    g.p.E = 1;
    g.p.J = N;
    g.p.C = K;
    g.p.out = out;
    g.p.bias = static_cast<const uint16_t*>(bias);
    g.p.residual = static_cast<const uint16_t*>(residual);
    g.p.pre = static_cast<uint16_t*>(pre);
    g.p.fn = fn;
    g.p.err = err_word;
    g.p.wait_ns = moe::wait_limit_ns();
    g.a = a;
    g.w = w;
    g.act = act;
    g.N = N;
    g.K = K;
    g.st = static_cast<cudaStream_t>(stream);
    g.who = who;
    return moe::launch_rows(g);
}
