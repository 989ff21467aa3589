// Forward products of the dense operators with e4m3 operands.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

bool run_e4m3_product(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPart)
    return p.gated ? launch_cfg<kKK, kE4m3, true, kEpiPart, float, false>(p, s)
                   : launch_cfg<kKK, kE4m3, false, kEpiPart, float, false>(p, s);
  return p.gated ? launch_cfg<kKK, kE4m3, true, kEpiFwd, __nv_bfloat16, false>(p, s)
                 : launch_cfg<kKK, kE4m3, false, kEpiFwd, __nv_bfloat16, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
