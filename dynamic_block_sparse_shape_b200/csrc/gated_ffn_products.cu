// The plain products of the feed-forward block.
#include "gated_ffn.h"

namespace prism {
prism_status ffn_product_nt(GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form) {
  return gemm<false, false, kEpiStore, 0>(P, &pr, 1, s, form);
}
prism_status ffn_product_nn(GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form) {
  return gemm<false, true, kEpiStore, 0>(P, &pr, 1, s, form);
}
prism_status ffn_products_tn(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s, GemmChoice* form) {
  return gemm<true, true, kEpiStore, 0>(P, pr, products, s, form);
}
}  // namespace prism
