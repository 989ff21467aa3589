// The softmax cross entropy's products: the logits twice (kEpiLse, kEpiXent),
// and dx added up over the pieces of the catalogue (kEpiAcc).
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

template <int EPI, bool F32>
bool launch_xent(const Product& p, cudaStream_t s) {
  return p.cfg == 0 ? launch_tc<2, cfg_bn(0, F32), kKK, kBf16, false, EPI, F32>(p, s)
                    : launch_tc<1, 128, kKK, kBf16, false, EPI, F32>(p, s);
}

bool run_xent_product(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiLse) return p.f32 ? launch_xent<kEpiLse, true>(p, s) : launch_xent<kEpiLse, false>(p, s);
  return p.f32 ? launch_xent<kEpiXent, true>(p, s) : launch_xent<kEpiXent, false>(p, s);
}

bool run_acc_product(const Product& p, cudaStream_t s) {
  return p.f32 ? launch_cfg<kKN, kBf16, false, kEpiAcc, true>(p, s) : launch_cfg<kKN, kBf16, false, kEpiAcc, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
