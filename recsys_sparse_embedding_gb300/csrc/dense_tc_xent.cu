// The softmax cross entropy's products: the logits twice (kEpiLse, kEpiXent),
// and dx added up over the pieces of the catalogue (kEpiAcc).
#include "dense_tc.cuh"
#include "xent_pass.cuh"

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

template <int MODE, int NK>
bool launch_pass(const PassArgs& a, const Mat& rows, const Mat& stream, cudaStream_t s) {
  auto* kernel = xent_pass_kernel<MODE, NK>;
  static std::atomic<int> grid_max[64];  // (host threads may race on it: each computes the same value)
  int dev = 0;
  if (!succeeded(cudaGetDevice(&dev)) || dev < 0 || dev >= 64) return false;
  int most = grid_max[dev].load(std::memory_order_acquire);
  if (most == 0) {
    if (!succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PassShape<NK>::SMEM)) ||
        !succeeded(cudaDeviceGetAttribute(&most, cudaDevAttrMultiProcessorCount, dev)) || most < 1)
      return false;
    grid_max[dev].store(most, std::memory_order_release);
  }
  CUtensorMap mr, ms;
  if (!tensor_map_3d(&mr, rows, 2, 64, 128) || !tensor_map_3d(&ms, stream, 2, 64, 128)) return false;
  const long long units = (long long)a.rt * a.chunks;
  if (units > INT32_MAX / 2) return false;
  return pdl_launch_smem(kernel, dim3(unsigned(units < most ? units : most)), PassShape<NK>::threads(MODE),
                         PassShape<NK>::SMEM, s, a, mr, ms);
}

template <int MODE>
bool run_pass(const PassArgs& a, const Mat& rows, const Mat& stream, cudaStream_t s) {
  return a.K <= 64 ? launch_pass<MODE, 1>(a, rows, stream, s) : launch_pass<MODE, 2>(a, rows, stream, s);
}

bool run_xent_pass(int mode, const PassArgs& a, const Mat& rows, const Mat& stream, cudaStream_t s) {
  return mode == kSums ? run_pass<kSums>(a, rows, stream, s)
                       : (mode == kDx ? run_pass<kDx>(a, rows, stream, s) : run_pass<kDw>(a, rows, stream, s));
}

}  // namespace dense
}  // namespace dsf
