// The product behind the gate's gradient in the feed-forward block's backward pass.
#include "gated_ffn.h"

namespace prism {
prism_status ffn_gate_bwd_product(int act, GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form) {
  switch (act) {
    case PRISM_ACT_SILU: return gemm<false, true, kEpiGateBwd, PRISM_ACT_SILU>(P, &pr, 1, s, form);
    case PRISM_ACT_GELU: return gemm<false, true, kEpiGateBwd, PRISM_ACT_GELU>(P, &pr, 1, s, form);
    case PRISM_ACT_GELU_TANH: return gemm<false, true, kEpiGateBwd, PRISM_ACT_GELU_TANH>(P, &pr, 1, s, form);
  }
  return gemm<false, true, kEpiGateBwd, PRISM_ACT_RELU>(P, &pr, 1, s, form);
}
}  // namespace prism
