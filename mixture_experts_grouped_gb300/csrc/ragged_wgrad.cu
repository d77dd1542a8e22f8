// Gradient form of the ragged products.
#include "ragged_tc.cuh"

namespace moe {
namespace ragged {
namespace {

template <int ACT, bool F32> int gradient_form(const RaggedArgs& g) {
    RaggedParams p = g.p;
    p.maxu = 256;
    CUtensorMap a, b, out;
    // of no rows, any address serves the maps: no copy is made
    const void* dy = p.rows ? g.a : p.out;
    const void* x = p.rows ? g.w : p.out;
    const uint64_t rows = p.rows ? p.rows : 1;
    int rc = make_tmap_2d(&a, dy, rows, p.J, 64, g.act);
    if (rc == MOE_OK) rc = make_tmap_2d(&b, x, rows, p.C, 64, g.act);
    if (rc == MOE_OK)
        rc = make_tmap_3d(&out, p.out, F32 ? kTmapF32 : g.act, p.C, p.J, p.E, F32 ? 32 : 64, 32);
    if (rc != MOE_OK) return rc;
    const int64_t tiles = static_cast<int64_t>(p.E) * ((p.J + 255) / 256) * ((p.C + p.maxu - 1) / p.maxu);
    return launch<WGRAD, ACT, F32, 1>(a, b, out, p, tiles, g.st, g.who);
}

}  // namespace
}  // namespace ragged

int launch_ragged_wgrad(const RaggedArgs& g) {
    if (g.act == MOE_ACT_BF16)
        return g.f32 ? ragged::gradient_form<MOE_ACT_BF16, true>(g) : ragged::gradient_form<MOE_ACT_BF16, false>(g);
    return g.f32 ? ragged::gradient_form<MOE_ACT_F16, true>(g) : ragged::gradient_form<MOE_ACT_F16, false>(g);
}

}  // namespace moe
