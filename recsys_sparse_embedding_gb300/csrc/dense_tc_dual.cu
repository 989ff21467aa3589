// The dense operators' backward: dx and dW in one launch, so that the units of
// one fill the last wave of the other.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

bool run_dual_product(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPart)
    return p.f32 ? launch_cfg<kDual, kBf16, false, kEpiPart, true>(p, s)
                 : launch_cfg<kDual, kBf16, false, kEpiPart, false>(p, s);
  return p.f32 ? launch_cfg<kDual, kBf16, false, kEpiOut, true>(p, s)
               : launch_cfg<kDual, kBf16, false, kEpiOut, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
