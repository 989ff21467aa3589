// Products that leave the next one's operand (the orthogonalised update): terms, or
// the terms of the Newton-Schulz polynomial.
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

template <int MAJOR, int EPI, bool TWO>
bool run_terms(const Product& p, cudaStream_t s) {
  if (p.cfg == 0) return launch_tc<2, cfg_bn(0, !TWO), MAJOR, kBf16, false, EPI, !TWO, TWO>(p, s);
  if (p.cfg == 1) return launch_tc<1, 128, MAJOR, kBf16, false, EPI, !TWO, TWO>(p, s);
  return launch_tc<1, 64, MAJOR, kBf16, false, EPI, !TWO, TWO>(p, s);
}
template <bool TWO>
bool run_any(const Product& p, cudaStream_t s) {
  if (p.epi == kEpiPoly) return run_terms<kKK, kEpiPoly, TWO>(p, s);
  return p.major == kKK ? run_terms<kKK, kEpiTerms, TWO>(p, s)
                        : (p.major == kKN ? run_terms<kKN, kEpiTerms, TWO>(p, s) : run_terms<kNN, kEpiTerms, TWO>(p, s));
}

bool run_terms_product(const Product& p, cudaStream_t s) { return p.two ? run_any<true>(p, s) : run_any<false>(p, s); }

}  // namespace dense
}  // namespace dsf
