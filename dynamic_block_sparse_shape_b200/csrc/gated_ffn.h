// The products of the feed-forward block, one call per kind (gated_ffn.cu
// puts them together; each kind is a source file of its own, so they compile
// side by side).
#pragma once
#include "gemm_host.cuh"

namespace prism {
// With `form` a product is not run: it says which kernel and tiles it takes.
// h = act(x Wg^T) (x Wu^T), with `save` also both projections
prism_status ffn_gate_product(int act, GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form);
// dh = dy Wd and from it dg, du, with `save` also h
prism_status ffn_gate_bwd_product(int act, GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form);
// both operands K-major / B MN-major / both MN-major
prism_status ffn_product_nt(GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form);
prism_status ffn_product_nn(GemmArgs& P, const GemmProblem& pr, cudaStream_t s, GemmChoice* form);
// Of at most kFineTokens tokens h, dg and du are held as bf16 values and, m rows
// further on, their bf16 remainders: the weights' bytes are the cost there.
constexpr int kFineTokens = 32;
// the whole forward pass of a handful of tokens, y = x allowed; h: [2 m, f]
bool ffn_takes_rows(int64_t m, int d);
prism_status ffn_rows_forward(int act, const prism_ffn_weights& w, int m, const void* x, int64_t x_ld, void* h, void* y,
                              int64_t y_ld, void* gate, void* up, cudaStream_t s);
prism_status ffn_products_tn(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s, GemmChoice* form);
}  // namespace prism
