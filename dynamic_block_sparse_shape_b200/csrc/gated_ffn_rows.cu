// The forward pass of the feed-forward block for a handful of tokens.
//
// The mathematics: dot products of weight rows with every token,
//   g_f = wg_f . x_m, u_f = wu_f . x_m, h_f = act(g_f) u_f,  then y_d = wd_d . h_m.
//
// What bounds it: the weights' bytes, read once (3 d f, at HBM's rate; a tile of
// the tensor cores would be empty but for a few rows, and its 128-byte pieces
// of 128 rows at a time reach 2 to 3 TB/s). So: fp32 multiply-adds on the
// ordinary cores, weights in 16-byte loads, whole rows in order. A CTA takes R
// weight rows; its warps take every eighth 256-value chunk of K, lane l the
// values 8 l .. 8 l + 7, with the tokens' values in registers for all R rows and
// the R loads of a chunk in flight together. Sums stay in fp32; lanes are
// added by butterflies and warps in shared memory in a fixed order.
// The down product's first weights are requested before it waits for h
// (programmatic dependent launch): they do not depend on it.
// 2048 x 5632, one token: see the table in the design notes for both kernels' times.
#include "gated_ffn.h"

namespace prism {
namespace {

constexpr int kRowWarps = 8;
constexpr int kRowChunk = 256;  // values of K per warp and step

struct RowArgs {
  const __nv_bfloat16* w[2];  // gate: Wg, Wu; down: Wd
  int64_t w_ld[2];
  const __nv_bfloat16* x;  // [m, k]
  int64_t x_ld;
  __nv_bfloat16* out[3];  // gate: h, g, u; down: y
  int64_t out_ld[3];
  int m, rows, k;  // rows: f or d
  int save;
};

// GATE: R / 2 rows of Wg, then the same of Wu; else R rows.
template <int M, int R, bool GATE, int ACT>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const RowArgs P) {
  constexpr int kOut = GATE ? R / 2 : R;  // output columns of a CTA
  __shared__ float part[kRowWarps][R * M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f0 = blockIdx.x * kOut;
  const __nv_bfloat16* row[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = GATE ? r / kOut : 0;
    const int f = min(f0 + r % kOut, P.rows - 1);  // rows behind the last repeat it and are not written
    row[r] = P.w[i] + f * P.w_ld[i];
  }
  float acc[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[r][m] = 0.f;
  int k = warp * kRowChunk + lane * 8;
  uint4 w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = k < P.k ? __ldg(reinterpret_cast<const uint4*>(row[r] + k)) : make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  grid_launch_dependents();
  for (; k < P.k; k += kRowWarps * kRowChunk) {
    // the next step's weights are on their way while this one is added
    const int next = k + kRowWarps * kRowChunk;
    uint4 wn[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      wn[r] = next < P.k ? __ldg(reinterpret_cast<const uint4*>(row[r] + next)) : make_uint4(0, 0, 0, 0);
    float x[M][8];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint4 v = m < P.m ? *reinterpret_cast<const uint4*>(P.x + m * P.x_ld + k) : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[m][2 * i] = __uint_as_float(u[i] << 16);
        x[m][2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t u[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xFFFF0000u);
#pragma unroll
        for (int m = 0; m < M; ++m) acc[r][m] = fmaf(hi, x[m][2 * i + 1], fmaf(lo, x[m][2 * i], acc[r][m]));
      }
      w[r] = wn[r];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float s = acc[r][m];
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) part[warp][r * M + m] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kOut * M; i += kRowWarps * 32) {
    const int r = i / M, m = i - r * M, f = f0 + r;
    if (f >= P.rows || m >= P.m) continue;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int v = 0; v < kRowWarps; ++v) {
      a += part[v][r * M + m];
      if constexpr (GATE) b += part[v][(r + kOut) * M + m];
    }
    if constexpr (GATE) {
      P.out[0][m * P.out_ld[0] + f] = __float2bfloat16_rn(act_f<ACT>(a) * b);
      if (P.save) {
        P.out[1][m * P.out_ld[1] + f] = __float2bfloat16_rn(a);
        P.out[2][m * P.out_ld[2] + f] = __float2bfloat16_rn(b);
      }
    } else {
      P.out[0][m * P.out_ld[0] + f] = __float2bfloat16_rn(a);
    }
  }
}

template <int M, bool GATE, int ACT>
prism_status launch_rows(const RowArgs& a, bool follows, cudaStream_t s) {
  constexpr int R = M <= 4 ? 8 : 4;  // R M sums and 8 M values of x in registers
  constexpr int kOut = GATE ? R / 2 : R;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((a.rows + kOut - 1) / kOut);
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = follows ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, rows_kernel<M, R, GATE, ACT>, a));
}

template <bool GATE, int ACT>
prism_status rows_for(const RowArgs& a, bool follows, cudaStream_t s) {
  if (a.m == 1) return launch_rows<1, GATE, ACT>(a, follows, s);
  if (a.m == 2) return launch_rows<2, GATE, ACT>(a, follows, s);
  if (a.m <= 4) return launch_rows<4, GATE, ACT>(a, follows, s);
  return launch_rows<8, GATE, ACT>(a, follows, s);
}

}  // namespace

prism_status ffn_rows_forward(int act, const prism_ffn_weights& w, int m, const void* x, int64_t x_ld, void* h, void* y,
                              int64_t y_ld, void* gate, void* up, cudaStream_t s) {
  using B = __nv_bfloat16;
  RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.w[0] = static_cast<const B*>(w.w_gate);
  a.w[1] = static_cast<const B*>(w.w_up);
  a.w_ld[0] = w.gate_stride;
  a.w_ld[1] = w.up_stride;
  a.x = static_cast<const B*>(x);
  a.x_ld = x_ld;
  void* out[3] = {h, gate, up};
  for (int i = 0; i < 3; ++i) {
    a.out[i] = static_cast<B*>(out[i]);
    a.out_ld[i] = w.f;
  }
  a.m = m; a.rows = w.f; a.k = w.d;
  a.save = gate != nullptr;
  prism_status st;
  switch (act) {
    case PRISM_ACT_SILU: st = rows_for<true, PRISM_ACT_SILU>(a, false, s); break;
    case PRISM_ACT_GELU: st = rows_for<true, PRISM_ACT_GELU>(a, false, s); break;
    case PRISM_ACT_GELU_TANH: st = rows_for<true, PRISM_ACT_GELU_TANH>(a, false, s); break;
    default: st = rows_for<true, PRISM_ACT_RELU>(a, false, s);
  }
  if (st != PRISM_OK) return st;
  a.w[0] = static_cast<const B*>(w.w_down);
  a.w_ld[0] = w.down_stride;
  a.x = static_cast<const B*>(h);
  a.x_ld = w.f;
  a.out[0] = static_cast<B*>(y);
  a.out_ld[0] = y_ld;
  a.rows = w.d; a.k = w.f;
  return rows_for<false, PRISM_ACT_SILU>(a, true, s);
}

}  // namespace prism
