// The dense operators' backward: dx = dz W (W MN-major) and dW = dz^T x (both
// operands MN-major), from the matrices as they are stored.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

template <int MAJOR>
bool run(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPart)
    return p.f32 ? launch_cfg<MAJOR, kBf16, false, kEpiPart, true>(p, s)
                 : launch_cfg<MAJOR, kBf16, false, kEpiPart, false>(p, s);
  return p.f32 ? launch_cfg<MAJOR, kBf16, false, kEpiOut, true>(p, s)
               : launch_cfg<MAJOR, kBf16, false, kEpiOut, false>(p, s);
}

bool run_grad_product(const Product& p, cudaStream_t s) { return p.major == kKN ? run<kKN>(p, s) : run<kNN>(p, s); }

}  // namespace dense
}  // namespace dsf
