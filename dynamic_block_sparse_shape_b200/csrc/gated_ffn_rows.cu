// The forward pass of the feed-forward block for a handful of tokens.
//
// The mathematics: dot products of weight rows with every token,
//   g_f = wg_f . x_m, u_f = wu_f . x_m, h_f = act(g_f) u_f,  then y_d = wd_d . h_m.
//
// What bounds it: the weights' bytes, read once (3 d f, at HBM's rate). Tiles of
// 128 rows by TMA fetch them in pieces of 128 bytes of 128 rows at a time, an SM
// at most 90 GB/s; here every SM streams whole rows. A CTA takes 16 weight rows
// (the gate product: 16 of Wg and the same 16 of Wu); its warps take blocks of K
// in turn, with the next block's loads under way while one is multiplied. The products are warp-wide m16n8k16: a lane's 16 bytes of a row
// are four pairs of k, and since the sum over k may go in any order, the pairs go
// into the instruction as they lie: tokens are read with the same permutation,
// and no value moves between lanes. Sums stay in fp32 and are added over the
// warps in shared memory in a fixed order. The gate product leaves h as m rows of
// bf16 values and m rows of their bf16 remainders; the down product takes them as
// 2 m tokens and adds the two, so y is rounded once and not on top of a rounded h.
// 2048 x 5632, cold weights: 1 and 4 tokens 18.3 us, 8 tokens 20.8, 16 24.0 in both
// launches (the tiles of the split kernel: 25 to 26; multiply-adds on the ordinary
// cores: 18.8 for one token, 45 for 8). h rounded to bf16 instead: 18.2 for one
// token, 19.0 for 8, 23.2 for 16, with 1.41 times the error of y; h in fp32, split
// as it is read: 20.3 and 29.4 for 1 and 16.
// The down product's first weights are requested before it waits for h
// (programmatic dependent launch): they do not depend on it.
#include "gated_ffn.h"

namespace prism {
namespace {

constexpr int kRowTile = 16;   // weight rows of a product

struct RowArgs {
  const __nv_bfloat16* w[2];  // gate: Wg, Wu; down: Wd
  int64_t w_ld[2];
  const __nv_bfloat16* x;  // [m, k]; down: h, [2 m, k]
  int64_t x_ld;
  __nv_bfloat16* out[3];  // gate: h, g, u; down: y
  int64_t out_ld;
  int m, rows, k;  // m: tokens of x (down: 2 m); rows: f or d
  int save;
};

__device__ __forceinline__ void mma_rows(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens; U: steps of 32 values of K whose loads go together.
template <int NT, bool GATE, int ACT, int U, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) rows_kernel(const RowArgs P) {
  constexpr int kRowWarps = WARPS, kU = U, kRowBlock = 32 * U;
  constexpr int kT = GATE ? 2 : 1;  // weight tiles
  __shared__ float part[kRowWarps][kT * kRowTile][NT * 8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // of the instruction's fragments: row or token, and k pair
  const int f0 = blockIdx.x * kRowTile;
  const __nv_bfloat16* row[kT][2];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows behind the last repeat it and are not written
      row[i][h] = P.w[i] + min(f0 + g + 8 * h, P.rows - 1) * P.w_ld[i] + 8 * t;
  const __nv_bfloat16* tok[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) tok[n] = P.x + min(8 * n + g, P.m - 1) * P.x_ld + 8 * t;
  float acc[kT][NT][4] = {};
  uint4 w[kU][kT][2];
  auto load = [&](int k, uint4 (&to)[kU][kT][2]) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          to[u][i][h] = k + 32 * u + 8 * t < P.k ? __ldg(reinterpret_cast<const uint4*>(row[i][h] + k + 32 * u))
                                                 : make_uint4(0, 0, 0, 0);
  };
  int k = warp * kRowBlock;
  load(k, w);
  grid_dependency_wait();
  grid_launch_dependents();
  for (; k < P.k; k += kRowWarps * kRowBlock) {
    uint4 next[kU][kT][2];
    load(k + kRowWarps * kRowBlock, next);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 x = k + 32 * u + 8 * t < P.k ? *reinterpret_cast<const uint4*>(tok[n] + k + 32 * u)
                                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          mma_rows(acc[i][n], w[u][i][0].x, w[u][i][1].x, w[u][i][0].y, w[u][i][1].y, x.x, x.y);
          mma_rows(acc[i][n], w[u][i][0].z, w[u][i][1].z, w[u][i][0].w, w[u][i][1].w, x.z, x.w);
        }
      }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[u][i][h] = next[u][i][h];
  }
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][i * kRowTile + g + 8 * (e >> 1)][8 * n + 2 * t + (e & 1)] = acc[i][n][e];
  __syncthreads();
  for (int x = threadIdx.x; x < kRowTile * NT * 8; x += kRowWarps * 32) {
    const int r = x % kRowTile, m = x / kRowTile, f = f0 + r;
    const int tokens = GATE ? P.m : P.m / 2;
    if (f >= P.rows || m >= tokens) continue;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int v = 0; v < kRowWarps; ++v) {
      a += part[v][r][m];
      b += GATE ? part[v][r + kRowTile][m] : part[v][r][m + tokens];
    }
    if constexpr (GATE) {
      const float h = act_f<ACT>(a) * b;
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      P.out[0][m * P.out_ld + f] = hi;
      P.out[0][(m + P.m) * P.out_ld + f] = __float2bfloat16_rn(remainder_bf16(h, __bfloat162float(hi)));
      if (P.save) {
        P.out[1][m * P.out_ld + f] = __float2bfloat16_rn(a);
        P.out[2][m * P.out_ld + f] = __float2bfloat16_rn(b);
      }
    } else {
      P.out[0][m * P.out_ld + f] = __float2bfloat16_rn(a + b);
    }
  }
}

template <int NT, bool GATE, int ACT, int U, int WARPS>
prism_status launch_rows_as(const RowArgs& a, bool follows, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((a.rows + kRowTile - 1) / kRowTile);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = follows ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, rows_kernel<NT, GATE, ACT, U, WARPS>, a));
}

// With a CTA per SM at most, K is shared by 16 warps, else by 4 that leave the SM
// room for other CTAs (the gate product of 1024 values of f, d = 4096: 11.2 us the
// call, 18.3 with 4). The down product has few rows and a long K: always 16, and
// with a CTA per SM at most 128 values at a time keep more loads in flight (2048 x
// 5632, one token: 9.8 us, 13.0 with 64); with more CTAs their registers count
// (4096 x 11264: 26.5 us, 22.7 with 64).
template <int NT, bool GATE, int ACT>
prism_status launch_rows(const RowArgs& a, bool follows, cudaStream_t s) {
  const bool few = (a.rows + kRowTile - 1) / kRowTile <= device_sm_count();
  if constexpr (GATE) {
    if (!few) return launch_rows_as<NT, GATE, ACT, 2, 4>(a, follows, s);
  } else {
    if (few) return launch_rows_as<NT, GATE, ACT, 4, 16>(a, follows, s);
  }
  return launch_rows_as<NT, GATE, ACT, 2, 16>(a, follows, s);
}

template <bool GATE, int ACT>
prism_status rows_for(const RowArgs& a, bool follows, cudaStream_t s) {
  if (a.m <= 8) return launch_rows<1, GATE, ACT>(a, follows, s);
  if constexpr (!GATE) {
    // few weight rows alone: see ffn_takes_rows
    if (a.m > 16) return launch_rows_as<4, GATE, ACT, 4, 16>(a, follows, s);
  }
  return launch_rows<2, GATE, ACT>(a, follows, s);
}

}  // namespace

// Up to 8 tokens, and up to 16 where a CTA per SM at most takes the down product:
// each reads all of h, by then more than its weights. 16 tokens, this way / by
// tiles: 1024 x 2816 13.3 / 15.5 us, 2048 x 5632 24.2 / 24.8, 2368 x 6400 28.9 /
// 29.3, 2384 x 6400 49.4 / 29.8, 4096 x 11264 104 / 63; 8 tokens: 2048 x 5632 20.7
// / 25.8, 4096 x 11264 52 / 63, 8192 x 22528 186 / 198.
bool ffn_takes_rows(int64_t m, int d) { return m <= 8 || (m <= 16 && (d + kRowTile - 1) / kRowTile <= device_sm_count()); }

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
  a.out[0] = static_cast<B*>(h);
  a.out[1] = static_cast<B*>(gate);
  a.out[2] = static_cast<B*>(up);
  a.out_ld = w.f;
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
  a.out_ld = y_ld;
  a.m = 2 * m; a.rows = w.d; a.k = w.f;
  return rows_for<false, PRISM_ACT_SILU>(a, true, s);
}

}  // namespace prism
