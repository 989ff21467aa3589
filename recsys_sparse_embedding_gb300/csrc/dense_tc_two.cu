// Products of operands in two bf16 terms (the orthogonalised update of bf16
// matrices): fp32 partial sums, operands K-major or MN-major.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

template <int MAJOR>
bool run_two(const Product& p, cudaStream_t s) {
  if (p.cfg == 0) return launch_tc<2, 256, MAJOR, kBf16, false, kEpiPart, false, true>(p, s);
  if (p.cfg == 1) return launch_tc<1, 128, MAJOR, kBf16, false, kEpiPart, false, true>(p, s);
  return launch_tc<1, 64, MAJOR, kBf16, false, kEpiPart, false, true>(p, s);
}

bool run_two_product(const Product& p, cudaStream_t s) {
  return p.major == kKK ? run_two<kKK>(p, s) : (p.major == kKN ? run_two<kKN>(p, s) : run_two<kNN>(p, s));
}

}  // namespace dense
}  // namespace dsf
