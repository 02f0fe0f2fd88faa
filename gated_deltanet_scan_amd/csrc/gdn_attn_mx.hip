// Softmax attention over block-scaled keys and values (MXFP8, MXFP4): the
// launches of gdn_attn_fwd_fp8 and gdn_attn_fwd_fp4.  The forward kernel is that
// of bf16 keys (gdn_attn_tile.hpp); codes are widened to bf16 as they are staged.
#include "gdn_attn_tile.hpp"

namespace gdnattn {
namespace {

template <typename F, int D, int NW>
gdn_status launch(AttnArgs a, Grid g, hipStream_t s) {
    a.tiles = g.tiles;
    hipLaunchKernelGGL((attn_fwd_kernel<KeysMx<F>, D, NW>), dim3(g.groups), dim3(64 * NW), 0, s, a);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
template <typename F>
gdn_status by_size(const AttnArgs& a, int rows, Grid g, hipStream_t s) {
    if (a.D == 32) return launch<F, 32, 4>(a, g, s);
    if (a.D == 64) return launch<F, 64, 4>(a, g, s);
    return rows == 256 ? launch<F, 128, 8>(a, g, s) : launch<F, 128, 4>(a, g, s);
}

}  // namespace

gdn_status attn_fwd_mx(const AttnArgs& a, bool fp4, int rows, Grid g, hipStream_t s) {
    return fp4 ? by_size<gdnmx::Fp4>(a, rows, g, s) : by_size<gdnmx::Fp8>(a, rows, g, s);
}

}  // namespace gdnattn
