// The dense operators' backward: z computed again and dz = dy act'(z) in the
// product's epilogue.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

bool run_dz_product(const Product& p, cudaStream_t s) {
  if (p.f32)
    return p.gated ? launch_cfg<kKK, kBf16, true, kEpiDz, true>(p, s)
                   : launch_cfg<kKK, kBf16, false, kEpiDz, true>(p, s);
  return p.gated ? launch_cfg<kKK, kBf16, true, kEpiDz, false>(p, s)
                 : launch_cfg<kKK, kBf16, false, kEpiDz, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
