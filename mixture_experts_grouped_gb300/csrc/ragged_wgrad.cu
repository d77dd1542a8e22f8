// Gradient form of the ragged products.
#include "ragged_split.cuh"

namespace moe {
namespace ragged {
namespace {

template <int ACT, int KIND> int gradient_form(const RaggedArgs& g) {
    RaggedParams p = g.p;
    const int nt = (p.J + 255) / 256, kt = g.kt;
    p.kunit = gradient_unit(g.f32);
    const int units = (p.C + p.kunit - 1) / p.kunit;
    p.kleast = units / kt;
    p.kmore = units % kt;
    const int64_t tiles = static_cast<int64_t>(p.E) * nt * kt;
    if (tiles > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", g.who);
    p.kt.set(kt);
    p.per.set(nt * kt);
    Maps m;
    // of no rows, any address serves the maps: no copy is made
    const void* dy = p.rows ? g.a : p.out;
    const void* x = p.rows ? g.w : p.out;
    const uint64_t rows = p.rows ? p.rows : 1;
    const int out = in_16_bits(KIND) ? g.act : kTmapF32;
    const uint32_t cols = in_16_bits(KIND) ? 64 : 32;
    int rc = make_tmap_2d(&m.a, dy, rows, p.J, 64, g.act, true);
    if (rc == MOE_OK) rc = make_tmap_2d(&m.b, x, rows, p.C, 64, g.act, true);
    if (rc == MOE_OK) rc = make_tmap_2d(&m.ta, dy, rows, p.J, 16, g.act);
    if (rc == MOE_OK) rc = make_tmap_2d(&m.tb, x, rows, p.C, 16, g.act);
    if (rc == MOE_OK) rc = make_tmap_3d(&m.out, p.out, out, p.C, p.J, p.E, cols, 32);
    m.add = m.out;
    if (rc == MOE_OK && KIND == GADD)
        rc = make_tmap_3d(&m.add, const_cast<float*>(p.addend), out, p.C, p.J, p.E, cols, 32);
    if (rc != MOE_OK) return rc;
    return launch<WGRAD, ACT, KIND>(m, p, tiles, g.st, g.who);
}

template <int ACT> int by_kind(const RaggedArgs& g) {
    if (g.parts) {
        const int kt = (g.p.C + 127) / 128;
        const int64_t tiles = static_cast<int64_t>((g.p.J + 127) / 128) * kt;
        const bool chunks = (g.p.rows + 64 * g.parts - 1) / (64 * g.parts) > gradient_chunk(g.f32, ACT);
        if (g.f32)
            return chunks ? launch_split_kind<WGRAD, ACT, G32LONG>(g, tiles, kt, g.parts)
                          : launch_split_kind<WGRAD, ACT, G32>(g, tiles, kt, g.parts);
        return chunks ? launch_split_kind<WGRAD, ACT, G16LONG>(g, tiles, kt, g.parts)
                      : launch_split_kind<WGRAD, ACT, G16>(g, tiles, kt, g.parts);
    }
    if (!g.f32)
        return g.p.rows > 64 * gradient_chunk(false, ACT) ? gradient_form<ACT, G16LONG>(g) : gradient_form<ACT, G16>(g);
    if (!g.p.addend) return gradient_form<ACT, G32>(g);
    // Addends come by TMA, through warps of their own, where groups are short and the gradient is
    // bound by its bytes: 12288 rows of 64 groups, 2048 x 1408, 234 us (282 by the adding warps'
    // loads); 512 rows of one, 4096 x 4096, 32 (36). Above, where a group has several chunks, which
    // that form adds in tensor memory while the pair's MMAs stand still, by loads: 700 rows of one 38
    // (43), 8192 of 8, 4096 x 3584, 222 (277).
    return g.p.rows <= 576 * static_cast<int64_t>(g.p.E) ? gradient_form<ACT, GADD>(g) : gradient_form<ACT, G32ADD>(g);
}

}  // namespace
}  // namespace ragged

int launch_ragged_wgrad(const RaggedArgs& g) {
    return g.act == MOE_ACT_BF16 ? ragged::by_kind<MOE_ACT_BF16>(g) : ragged::by_kind<MOE_ACT_F16>(g);
}

}  // namespace moe
