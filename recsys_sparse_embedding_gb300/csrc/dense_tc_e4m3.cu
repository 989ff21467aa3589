// Forward products of the dense operators with e4m3 operands.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

bool run_e4m3_product(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPart)
    return p.gated ? launch_cfg<kKK, kE4m3, true, kEpiPart, false>(p, s)
                   : launch_cfg<kKK, kE4m3, false, kEpiPart, false>(p, s);
  if (p.epi == kEpiRes) return launch_cfg<kKK, kE4m3, false, kEpiRes, false>(p, s);
  return p.gated ? launch_cfg<kKK, kE4m3, true, kEpiFwd, false>(p, s)
                 : launch_cfg<kKK, kE4m3, false, kEpiFwd, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
