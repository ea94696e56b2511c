// The gated feed-forward block behind the attention of a layer:
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T,
// and its gradient at the saved g, u:
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g),
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h.
//
// Forward: two launches. Both projections, the activation and the product are
// one kernel: a tile's accumulator holds g and u of the same columns, the
// epilogue forms h from them in fp32 and rounds once; g and u are written only
// when they are wanted for the backward pass. Backward: three launches: dh
// stays in tensor memory and becomes dg, du (and h again, from the saved
// projections, so the forward need not keep it) in the epilogue; dx is one
// product over both halves of K; the three weight gradients share a launch.
// dg, du and h are rounded to bf16 once each, as operands of the next product;
// of at most kFineTokens tokens they carry their remainders along (twice the rows,
// or a second segment of K, where the weights' bytes are the cost), so that every
// output is rounded once.
// Tensor operations: 6 M D F forward, 12 M D F backward; gemm.cuh says what
// bounds the products.
#include "gated_ffn.h"

namespace prism {
namespace {

// Workspace: the status word, then h (forward), or dg, du, h (backward): [m, f]
// bf16, of few tokens [2 m, f] with the remainders behind.
size_t ffn_part_bytes(int64_t m, int64_t f) {
  return align_up(size_t(m) * size_t(f) * (m <= kFineTokens ? 4 : 2), 256);
}
size_t ffn_ws_bytes(int64_t m, int64_t f, bool backward) {
  return kWsHeader + size_t(backward ? 3 : 1) * ffn_part_bytes(m, f);
}

struct Rows {
  const void* p;
  int64_t ld, width;
};

prism_status check_ffn(int64_t m, int32_t d, int32_t f, int32_t act, prism_dtype dtype) {
  if (dtype != PRISM_BF16) return PRISM_ERR_DTYPE;
  if (act < PRISM_ACT_SILU || act > PRISM_ACT_RELU) return PRISM_ERR_ARG;
  if (m < 0 || d < 1 || f < 1) return PRISM_ERR_ARG;
  if (d % 8 || f % 8) return PRISM_ERR_UNSUPPORTED;
  if (m > (int64_t(1) << 30) || d > (1 << 20) || f > (1 << 20)) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

prism_status check_rows(const Rows& r) {
  if (!r.p || reinterpret_cast<uintptr_t>(r.p) % 16) return PRISM_ERR_ARG;
  if (r.ld < r.width || r.ld % 8) return PRISM_ERR_ARG;
  if (r.ld >= (int64_t(1) << 31)) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

prism_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  return !ws || reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < need ? PRISM_ERR_WORKSPACE : PRISM_OK;
}

// Address ranges of a written and another tensor may not meet.
bool meet(const void* a, int64_t lda, int64_t na, int64_t wa, const void* b, int64_t ldb, int64_t nb, int64_t wb) {
  if (!a || !b || na < 1 || nb < 1) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + uintptr_t((na - 1) * lda + wa) * 2, b1 = b0 + uintptr_t((nb - 1) * ldb + wb) * 2;
  return a0 < b1 && b0 < a1;
}

// `bytes` of the workspace, which every launch writes and reads, and a tensor.
bool meet_ws(const void* ws, size_t bytes, const void* b, int64_t ldb, int64_t nb, int64_t wb) {
  return meet(ws, 0, 1, int64_t(bytes / 2), b, ldb, nb, wb);
}

// The launches of a checked call; with `form` none, but what each would take.
prism_status run_fwd(const prism_ffn_weights& w, int64_t m, int32_t act, const void* x, int64_t x_stride, void* y,
                     int64_t y_stride, void* gate, void* up, void* ws, cudaStream_t s, GemmChoice* form) {
  const int32_t d = w.d, f = w.f;
  prism_status st;
  void* h = static_cast<uint8_t*>(ws) + kWsHeader;
  if (ffn_takes_rows(m, d)) return form ? PRISM_OK : ffn_rows_forward(act, w, int(m), x, x_stride, h, y, y_stride, gate, up, s);
  GemmArgs P;
  std::memset(&P, 0, sizeof(P));
  P.status = ws_status(ws);
  P.save = gate != nullptr;
  GemmProblem g;
  g.a[0] = {x, x_stride};
  g.b[0] = {w.w_gate, w.gate_stride};
  g.b[1] = {w.w_up, w.up_stride};
  g.out[0] = {h, f};
  g.out[1] = {gate, f};
  g.out[2] = {up, f};
  g.m = m; g.n = f; g.k[0] = d;
  const bool fine = m <= kFineTokens;
  P.fine = fine;
  if ((st = ffn_gate_product(act, P, g, s, form)) != PRISM_OK) return st;
  GemmProblem r;
  r.a[0] = {h, f};
  r.b[0] = {w.w_down, w.down_stride};
  r.out[0] = {y, y_stride};
  r.m = fine ? 2 * m : m;  // the values' rows, then the remainders': added to one another at the end
  r.n = d; r.k[0] = f;
  P.follows = 1;
  P.fine = 0;
  P.fold = fine ? int(m) : 0;
  return ffn_product_nt(P, r, s, form ? form + 1 : nullptr);
}

prism_status run_bwd(const prism_ffn_weights& w, int64_t m, int32_t act, const void* dy, int64_t dy_stride, const void* x,
                     int64_t x_stride, const void* gate, const void* up, void* dx, int64_t dx_stride, void* dw_gate,
                     void* dw_up, void* dw_down, void* ws, cudaStream_t s, GemmChoice* form) {
  const int32_t d = w.d, f = w.f;
  const bool dw = dw_gate != nullptr;
  prism_status st;
  const size_t part = ffn_part_bytes(m, f);
  const bool fine = m <= kFineTokens;
  uint8_t* base = static_cast<uint8_t*>(ws) + kWsHeader;
  void *dg = base, *du = base + part, *h = base + 2 * part;
  GemmArgs P;
  std::memset(&P, 0, sizeof(P));
  P.status = ws_status(ws);
  P.save = dw;
  GemmProblem g;
  g.a[0] = {dy, dy_stride};
  g.in[0] = gate;
  g.in[1] = up;
  g.b[0] = {w.w_down, w.down_stride};
  g.out[0] = {dg, f};
  g.out[1] = {du, f};
  g.out[2] = {h, f};
  g.m = m; g.n = f; g.k[0] = d;
  P.fine = fine;
  if ((st = ffn_gate_bwd_product(act, P, g, s, form)) != PRISM_OK) return st;
  P.follows = 1;
  P.fine = 0;
  if (dx) {
    GemmProblem r;
    r.a[0] = {dg, f};
    r.a[1] = {du, f};
    r.b[0] = {w.w_gate, w.gate_stride};
    r.b[1] = {w.w_up, w.up_stride};
    r.out[0] = {dx, dx_stride};
    r.m = fine ? 2 * m : m;  // folded as in the forward
    r.n = d; r.k[0] = f; r.k[1] = f;
    P.fold = fine ? int(m) : 0;
    if ((st = ffn_product_nn(P, r, s, form ? form + 1 : nullptr)) != PRISM_OK) return st;
    P.fold = 0;
  }
  if (dw) {
    GemmProblem r[3];
    const void* a[3] = {dg, du, dy};
    void* o[3] = {dw_gate, dw_up, dw_down};
    for (int i = 0; i < 3; ++i) {
      r[i].a[0] = {a[i], i < 2 ? f : dy_stride};
      r[i].b[0] = {i < 2 ? x : h, i < 2 ? x_stride : f};
      r[i].out[0] = {o[i], i < 2 ? d : f};
      r[i].m = i < 2 ? f : d;
      r[i].n = i < 2 ? d : f;
      r[i].k[0] = m;
      if (fine) {  // the remainders as a second segment of K
        const int64_t below = m * f;
        r[i].a[1] = r[i].a[0];
        r[i].b[1] = r[i].b[0];
        GemmOperand& o2 = i < 2 ? r[i].a[1] : r[i].b[1];
        o2.base = static_cast<const __nv_bfloat16*>(o2.base) + below;
        r[i].k[1] = m;
      }
    }
    P.beside = dx != nullptr;
    if ((st = ffn_products_tn(P, r, 3, s, form ? form + 2 : nullptr)) != PRISM_OK) return st;
  }
  return PRISM_OK;
}

}  // namespace
}  // namespace prism

using namespace prism;

extern "C" prism_status prism_gated_ffn_workspace_size(int64_t m, int32_t f, int32_t backward, size_t* bytes) {
  if (!bytes || m < 0 || f < 1) return PRISM_ERR_ARG;
  if (m > (int64_t(1) << 30) || f > (1 << 20)) return PRISM_ERR_UNSUPPORTED;
  *bytes = ffn_ws_bytes(m, f, backward != 0);
  return PRISM_OK;
}

extern "C" prism_status prism_gated_ffn_fwd(const prism_ffn_weights* w, int64_t m, int32_t act, prism_dtype dtype,
                                            const void* x, int64_t x_stride, void* y, int64_t y_stride, void* gate,
                                            void* up, void* ws, size_t ws_bytes, void* stream) {
  if (!w) return PRISM_ERR_ARG;
  const int32_t d = w->d, f = w->f;
  prism_status st = check_ffn(m, d, f, act, dtype);
  if (st != PRISM_OK) return st;
  const Rows rows[] = {{w->w_gate, w->gate_stride, d}, {w->w_up, w->up_stride, d}, {w->w_down, w->down_stride, f}};
  for (const Rows& r : rows)
    if ((st = check_rows(r)) != PRISM_OK) return st;
  if (m > 0) {
    if ((st = check_rows({x, x_stride, d})) != PRISM_OK || (st = check_rows({y, y_stride, d})) != PRISM_OK) return st;
  }
  if (!gate != !up) return PRISM_ERR_ARG;
  if (gate && (reinterpret_cast<uintptr_t>(gate) % 16 || reinterpret_cast<uintptr_t>(up) % 16)) return PRISM_ERR_ARG;
  const size_t need = ffn_ws_bytes(m, f, false);
  if ((st = check_ws(ws, ws_bytes, need)) != PRISM_OK) return st;
  // what the first launch writes is not among what either reads, y not among what the first writes or the weights
  for (const void* o : {static_cast<const void*>(gate), static_cast<const void*>(up)}) {
    if (meet(o, f, m, f, x, x_stride, m, d) || meet(o, f, m, f, y, y_stride, m, d)) return PRISM_ERR_ARG;
    for (int i = 0; i < 3; ++i)
      if (meet(o, f, m, f, rows[i].p, rows[i].ld, i < 2 ? f : d, rows[i].width)) return PRISM_ERR_ARG;
  }
  if (meet(gate, f, m, f, up, f, m, f)) return PRISM_ERR_ARG;
  for (int i = 0; i < 3; ++i) {
    const int64_t n = i < 2 ? f : d;
    if (meet(y, y_stride, m, d, rows[i].p, rows[i].ld, n, rows[i].width)) return PRISM_ERR_ARG;
    if (meet_ws(ws, need, rows[i].p, rows[i].ld, n, rows[i].width)) return PRISM_ERR_ARG;
  }
  if (meet_ws(ws, need, x, x_stride, m, d) || meet_ws(ws, need, y, y_stride, m, d)) return PRISM_ERR_ARG;
  if (meet_ws(ws, need, gate, f, m, f) || meet_ws(ws, need, up, f, m, f)) return PRISM_ERR_ARG;
  if (m == 0) return PRISM_OK;
  return run_fwd(*w, m, act, x, x_stride, y, y_stride, gate, up, ws, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

extern "C" prism_status prism_gated_ffn_bwd(const prism_ffn_weights* w, int64_t m, int32_t act, prism_dtype dtype,
                                            const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                            const void* gate, const void* up, void* dx, int64_t dx_stride,
                                            void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                            void* stream) {
  if (!w) return PRISM_ERR_ARG;
  const int32_t d = w->d, f = w->f;
  prism_status st = check_ffn(m, d, f, act, dtype);
  if (st != PRISM_OK) return st;
  const Rows wr[] = {{w->w_gate, w->gate_stride, d}, {w->w_up, w->up_stride, d}, {w->w_down, w->down_stride, f}};
  for (const Rows& r : wr)
    if ((st = check_rows(r)) != PRISM_OK) return st;
  const bool dw = dw_gate || dw_up || dw_down;
  if (dw && !(dw_gate && dw_up && dw_down)) return PRISM_ERR_ARG;
  if (m > 0 && !dx && !dw) return PRISM_ERR_ARG;
  for (const void* p : {dw_gate, dw_up, dw_down})
    if (reinterpret_cast<uintptr_t>(p) % 16) return PRISM_ERR_ARG;
  if (m > 0) {
    const Rows rows[] = {{dy, dy_stride, d}, {x, x_stride, d}, {gate, f, f}, {up, f, f}};
    for (const Rows& r : rows)
      if ((st = check_rows(r)) != PRISM_OK) return st;
    if (dx && (st = check_rows({dx, dx_stride, d})) != PRISM_OK) return st;
  }
  const size_t need = ffn_ws_bytes(m, f, true);
  if ((st = check_ws(ws, ws_bytes, need)) != PRISM_OK) return st;
  {
    // no output over an input or another output, and nothing over the workspace
    const struct {
      const void* p;
      int64_t ld, n, width;
    } t[] = {{dx, dx_stride, m, d}, {dw_gate, d, f, d}, {dw_up, d, f, d}, {dw_down, f, d, f},  // written
             {dy, dy_stride, m, d}, {x, x_stride, m, d}, {gate, f, m, f}, {up, f, m, f},
             {w->w_gate, w->gate_stride, f, d}, {w->w_up, w->up_stride, f, d}, {w->w_down, w->down_stride, d, f}};
    for (int i = 0; i < 4; ++i)
      for (int j = i + 1; j < 11; ++j)
        if (meet(t[i].p, t[i].ld, t[i].n, t[i].width, t[j].p, t[j].ld, t[j].n, t[j].width)) return PRISM_ERR_ARG;
    for (const auto& r : t)
      if (meet_ws(ws, need, r.p, r.ld, r.n, r.width)) return PRISM_ERR_ARG;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (m == 0) {  // sums over no token
    for (void* p : {dw_gate, dw_up, dw_down})
      if (p && cudaMemsetAsync(p, 0, size_t(d) * f * 2, s) != cudaSuccess) return PRISM_ERR_CUDA;
    return PRISM_OK;
  }
  return run_bwd(*w, m, act, dy, dy_stride, x, x_stride, gate, up, dx, dx_stride, dw_gate, dw_up, dw_down, ws, s, nullptr);
}

extern "C" prism_status prism_gated_ffn_forms(const prism_ffn_weights* w, int64_t m, int32_t backward, int32_t* forms) {
  if (!w || !forms) return PRISM_ERR_ARG;
  const prism_status st = check_ffn(m, w->d, w->f, PRISM_ACT_SILU, PRISM_BF16);
  if (st != PRISM_OK) return st;
  std::memset(forms, 0, sizeof(int32_t) * 9);
  if (m == 0) return PRISM_OK;
  GemmChoice c[3] = {};
  alignas(16) char any[1];  // marks outputs that are wanted; nothing is launched
  const int64_t d = w->d;
  if (backward)
    run_bwd(*w, m, PRISM_ACT_SILU, any, d, any, d, any, any, any, d, any, any, any, any, nullptr, c);
  else
    run_fwd(*w, m, PRISM_ACT_SILU, any, d, any, d, any, any, any, nullptr, c);
  for (int i = 0; i < 3; ++i) {
    forms[3 * i] = c[i].cg;
    forms[3 * i + 1] = c[i].bn;
    forms[3 * i + 2] = c[i].parts;
  }
  return PRISM_OK;
}
