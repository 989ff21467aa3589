// Forward products of the dense operators (K-major bf16 operands), and the
// products' tensor maps.
#include <cudaTypedefs.h>

#include <mutex>

#include "dense_tc.cuh"

namespace dsf {
namespace dense {

namespace {
// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (succeeded(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q)) &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}
}  // namespace

// x as a 3-D tensor of esize-byte elements whose boxes are box_cols (128
// bytes, the swizzle span) by box_rows; reads past its edges give zeros.
bool tensor_map_3d(CUtensorMap* m, const Mat& x, int esize, int box_cols, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(x.cols), cuuint64_t(x.rows), cuuint64_t(x.planes)};
  const cuuint64_t strides[2] = {cuuint64_t(x.ld) * esize,
                                 cuuint64_t(x.planes > 1 ? x.plane : x.ld) * esize};
  const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1}, es[3] = {1, 1, 1};
  const CUtensorMapDataType t = esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return fn(m, t, 3, const_cast<void*>(x.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool run_fwd_product(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPart) {
    if (p.f32)
      return p.gated ? launch_cfg<kKK, kBf16, true, kEpiPart, true>(p, s)
                     : launch_cfg<kKK, kBf16, false, kEpiPart, true>(p, s);
    return p.gated ? launch_cfg<kKK, kBf16, true, kEpiPart, false>(p, s)
                   : launch_cfg<kKK, kBf16, false, kEpiPart, false>(p, s);
  }
  if (p.epi == kEpiRes)
    return p.f32 ? launch_cfg<kKK, kBf16, false, kEpiRes, true>(p, s) : launch_cfg<kKK, kBf16, false, kEpiRes, false>(p, s);
  if (p.f32)
    return p.gated ? launch_cfg<kKK, kBf16, true, kEpiFwd, true>(p, s)
                   : launch_cfg<kKK, kBf16, false, kEpiFwd, true>(p, s);
  return p.gated ? launch_cfg<kKK, kBf16, true, kEpiFwd, false>(p, s)
                 : launch_cfg<kKK, kBf16, false, kEpiFwd, false>(p, s);
}

}  // namespace dense
}  // namespace dsf
