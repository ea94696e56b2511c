// Rotary positions of Q and K, in the place where the block pooling, the
// scoring and the attention read them, and the transposed rotation of dQ and
// dK after the attention's backward pass.
//
// The mathematics. Pair i of a head (channels 2i, 2i + 1 interleaved, or i,
// i + rot/2 in halves) of the token at position p turns by the angle
//   a = (offset_x + p_x * scale_x) * f_i
// of its axis x (t, h, w of the token grid, or one given position):
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a).
// The transposed rotation (the gradient) is the same with -a. The frequencies
// f_i come from the host in 64 bits as turns per position (f_i / 2 pi), so a
// position anywhere in the int32 range keeps its fraction of a turn: the turn
// is one fp64 multiply-add, reduced to [-1/2, 1/2] in fp64, and only then
// rounded to fp32 (an error of 2^-25 turns at most) for sin and cos.
//
// What bounds it: HBM, every element read once and written once, three
// operations each. The angles depend on (token, pair) alone, so a CTA computes
// those of its few tokens once into shared memory (two values per pair) and
// every head of Q and K reads them from there; a thread keeps one vector's
// place inside the head and walks the heads, so its cosines and sines sit in
// registers per token and the loop has no divisions. kBatch vectors per thread
// are in flight before the first is used.
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "host.h"

namespace prism {
namespace {

constexpr int kRopeMaxHeadDim = 256;
constexpr int kRopeMaxPairs = kRopeMaxHeadDim / 2;
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 8;  // tokens per CTA
constexpr int kBatch = 4;

struct RopeArgs {
  const void* src[2];  // Q, K
  void* dst[2];
  int64_t src_ld[2], dst_ld[2];  // elements between tokens
  int64_t n;                     // tokens
  const int32_t* pos;            // [n, axes], or null: the raster grid
  int heads_q, heads;            // heads of Q, of both
  int head_dim, pairs;
  int axes;          // 1 or 3
  int pair1, pair2;  // first pair of axis 1, of axis 2
  int grid_h, grid_w;
  int rot_units, units;  // vectors (half: vector pairs) a head's rotated part has, and all that are touched
  int head_groups, token_groups, tokens;  // of a CTA
  float m, sign;
  double turn[kRopeMaxPairs];   // turns per position
  double start[kRopeMaxPairs];  // turns at position 0
};

// EV elements at an address aligned to their size.
template <typename T, int EV>
struct Vec {
  alignas(sizeof(T) * EV) T e[EV];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// HALF: a unit is two vectors of EV elements, rot/2 apart; otherwise one
// vector of EV elements, EV/2 pairs. EV is the widest vector that the sizes,
// strides and addresses allow (16 bytes on every usual layout). With ELEM the
// vector's elements are loaded and stored one by one (an interleaved pair at
// an address that is no multiple of its size).
template <typename T, int EV, bool HALF, bool ELEM>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs P) {
  extern __shared__ float2 cs[];  // [tokens][pairs]: m cos a, m sin a
  const int64_t n0 = int64_t(blockIdx.x) * P.tokens;
  for (int x = threadIdx.x; x < P.tokens * P.pairs; x += blockDim.x) {
    const int tok = x / P.pairs, i = x - tok * P.pairs;
    const int64_t n = n0 + tok;
    if (n >= P.n) break;
    const int axis = i < P.pair1 ? 0 : i < P.pair2 ? 1 : 2;
    int p;
    if (P.pos) {
      p = P.pos[n * P.axes + axis];
    } else if (P.axes == 1) {
      p = int(n);
    } else {
      const int r = int(n), row = r / P.grid_w;
      p = axis == 2 ? r - row * P.grid_w : axis == 1 ? row % P.grid_h : row / P.grid_h;
    }
    const double turns = fma(double(p), P.turn[i], P.start[i]);
    const float r = float(turns - rint(turns));
    float s, c;
    sincospif(2.f * r, &s, &c);
    cs[x] = make_float2(c * P.m, s * P.m * P.sign);
  }
  __syncthreads();
  const int group = threadIdx.x / P.units, u = threadIdx.x - group * P.units;
  const int tg = group / P.head_groups, hg = group - tg * P.head_groups;
  constexpr int kPairs = HALF ? EV : EV / 2;  // of a unit
  const bool rot = u < P.rot_units;
  // where the unit sits in the head, and its second vector (half layout)
  const int c0 = HALF && !rot ? 2 * P.rot_units * EV + (u - P.rot_units) * EV : u * EV;
  const int c1 = HALF && rot ? c0 + P.pairs : c0;
  // an interleaved vector may hold the last rotated pair and unrotated ones
  const int valid = rot ? min(kPairs, P.pairs - u * kPairs) : 0;
  using V = Vec<T, EV>;
  for (int tok = tg; tok < P.tokens; tok += P.token_groups) {
    const int64_t n = n0 + tok;
    if (n >= P.n) break;
    float co[kPairs], si[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 v = i < valid ? cs[tok * P.pairs + u * kPairs + i] : make_float2(1.f, 0.f);
      co[i] = v.x;
      si[i] = v.y;
    }
    for (int h0 = hg; h0 < P.heads; h0 += kBatch * P.head_groups) {
      V a[kBatch], b[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int h = h0 + j * P.head_groups;
        if (h < P.heads) {
          const int w = h >= P.heads_q;
          const T* s = static_cast<const T*>(P.src[w]) + n * P.src_ld[w] + int64_t(h - (w ? P.heads_q : 0)) * P.head_dim;
          if constexpr (ELEM) {
#pragma unroll
            for (int e = 0; e < EV; ++e) a[j].e[e] = s[c0 + e];
          } else {
            a[j] = *reinterpret_cast<const V*>(s + c0);
            if (HALF && rot) b[j] = *reinterpret_cast<const V*>(s + c1);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int h = h0 + j * P.head_groups;
        if (h < P.heads) {
          const int w = h >= P.heads_q;
          T* d = static_cast<T*>(P.dst[w]) + n * P.dst_ld[w] + int64_t(h - (w ? P.heads_q : 0)) * P.head_dim;
          if constexpr (HALF) {
            if (rot) {
#pragma unroll
              for (int e = 0; e < EV; ++e) {
                const float x = to_f(a[j].e[e]), y = to_f(b[j].e[e]);
                a[j].e[e] = from_f<T>(x * co[e] - y * si[e]);
                b[j].e[e] = from_f<T>(y * co[e] + x * si[e]);
              }
              *reinterpret_cast<V*>(d + c1) = b[j];
            }
          } else {
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
              if (e < valid) {  // the others keep their bits, NaN and infinities too
                const float x = to_f(a[j].e[2 * e]), y = to_f(a[j].e[2 * e + 1]);
                a[j].e[2 * e] = from_f<T>(x * co[e] - y * si[e]);
                a[j].e[2 * e + 1] = from_f<T>(y * co[e] + x * si[e]);
              }
            }
          }
          if constexpr (ELEM) {
#pragma unroll
            for (int e = 0; e < EV; ++e) d[c0 + e] = a[j].e[e];
          } else {
            *reinterpret_cast<V*>(d + c0) = a[j];
          }
        }
      }
    }
  }
}

// Turns per position of pair j of an axis with n rotated channels.
double pair_turns(const prism_rope_params& r, int n, int j) {
  const double two_pi = 6.283185307179586476925286766559;
  double theta = r.theta;
  if (r.scaling == PRISM_ROPE_NTK && n > 2) theta *= std::pow(r.factor, double(n) / (n - 2));
  const double f = std::pow(theta, -2.0 * j / n);
  double share = r.scaling == PRISM_ROPE_LINEAR ? 1.0 : 0.0;  // of the stretched frequency
  if (r.scaling == PRISM_ROPE_YARN) {
    // pairs that turn more than 32 times over the trained length keep their
    // frequency, those below one turn are stretched, a ramp over the index between
    const double per = n / (2.0 * std::log(theta));
    const double low = std::fmax(std::floor(per * std::log(r.trained_len / (32.0 * two_pi))), 0.0);
    const double high = std::fmin(std::ceil(per * std::log(r.trained_len / two_pi)), double(n - 1));
    share = std::fmin(std::fmax((j - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
  }
  return (f / r.factor * share + f * (1.0 - share)) / two_pi;
}

prism_status check_rope(const prism_rope_params* r, int head_dim, int* rot) {
  if (!r) return PRISM_ERR_ARG;
  if (r->layout != PRISM_ROPE_INTERLEAVED && r->layout != PRISM_ROPE_HALF) return PRISM_ERR_ARG;
  if (r->scaling < PRISM_ROPE_UNSCALED || r->scaling > PRISM_ROPE_YARN) return PRISM_ERR_ARG;
  if (r->n_axes != 1 && r->n_axes != 3) return PRISM_ERR_ARG;
  if (!(r->theta > 1.0) || !std::isfinite(r->theta) || !std::isfinite(r->magnitude)) return PRISM_ERR_ARG;
  if (r->scaling != PRISM_ROPE_UNSCALED && (!(r->factor > 0.0) || !std::isfinite(r->factor))) return PRISM_ERR_ARG;
  if (r->scaling == PRISM_ROPE_YARN && (!(r->trained_len > 0.0) || !std::isfinite(r->trained_len)))
    return PRISM_ERR_ARG;
  int64_t sum = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    if (r->axis_dim[a] < 0 || r->axis_dim[a] % 2) return PRISM_ERR_ARG;
    if (!std::isfinite(r->pos_scale[a]) || !std::isfinite(r->pos_offset[a])) return PRISM_ERR_ARG;
    sum += r->axis_dim[a];
  }
  if (head_dim < 2 || head_dim % 2 || head_dim > kRopeMaxHeadDim) return PRISM_ERR_UNSUPPORTED;
  if (sum < 2 || sum > head_dim) return PRISM_ERR_ARG;
  *rot = int(sum);
  return PRISM_OK;
}

// Do rows of `wa` bytes every `sa` bytes from a, and of `wb` every `sb` from
// b, n each, share memory? Exact for equal strides (views of one packed
// buffer); for different strides, whether the address ranges meet.
bool rows_meet(uintptr_t a, int64_t sa, int64_t wa, uintptr_t b, int64_t sb, int64_t wb, int64_t n) {
  const uintptr_t ea = a + uintptr_t((n - 1) * sa + wa), eb = b + uintptr_t((n - 1) * sb + wb);
  if (ea <= b || eb <= a) return false;
  if (sa != sb) return true;
  int64_t d = int64_t(b - a) % sa;
  if (d < 0) d += sa;
  return d < wa || d + wb > sa;
}

template <typename T, int EV, bool HALF, bool ELEM>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int64_t ctas = (a.n + a.tokens - 1) / a.tokens;
  const int threads = a.units * a.head_groups * a.token_groups;
  const size_t smem = size_t(a.tokens) * a.pairs * sizeof(float2);
  rope_kernel<T, EV, HALF, ELEM><<<unsigned(ctas), threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const RopeArgs& a, int ev, bool half, cudaStream_t s) {
  constexpr int kWide = 16 / int(sizeof(T));
  if (!half) {
    if (ev == kWide) return launch<T, kWide, false, false>(a, s);
    return launch<T, 2, false, true>(a, s);
  }
  if constexpr (kWide == 8) {
    if (ev == 8) return launch<T, 8, true, false>(a, s);
  }
  if (ev == 4) return launch<T, 4, true, false>(a, s);
  if (ev == 2) return launch<T, 2, true, false>(a, s);
  return launch<T, 1, true, false>(a, s);
}

}  // namespace
}  // namespace prism

using namespace prism;

extern "C" prism_status prism_rope(const prism_rope_params* params, const prism_dim3* grid, const int32_t* positions,
                                   int64_t n_tokens, const void* q, void* q_out, int32_t heads_q, int64_t q_stride,
                                   int64_t q_out_stride, const void* k, void* k_out, int32_t heads_k,
                                   int64_t k_stride, int64_t k_out_stride, prism_dtype dtype, int32_t head_dim,
                                   int32_t transposed, void* stream) {
  int rot = 0;
  prism_status st = check_rope(params, head_dim, &rot);
  if (st != PRISM_OK) return st;
  if (dtype != PRISM_BF16 && dtype != PRISM_FP32) return PRISM_ERR_DTYPE;
  if (n_tokens < 0) return PRISM_ERR_ARG;
  if (n_tokens > (int64_t(1) << 30)) return PRISM_ERR_UNSUPPORTED;
  if (!positions && params->n_axes == 3) {
    if (!grid || grid->t < 0 || grid->h < 0 || grid->w < 0) return PRISM_ERR_ARG;
    if ((grid->t > 0 && grid->h > 0 && int64_t(grid->t) * grid->h > (int64_t(1) << 30)) ||
        int64_t(grid->t) * grid->h * grid->w != n_tokens)
      return PRISM_ERR_SHAPE;
  }
  if (reinterpret_cast<uintptr_t>(positions) % 4) return PRISM_ERR_ARG;
  const int hk = k ? heads_k : 0;
  if (heads_q < 1 || (k && heads_k < 1)) return PRISM_ERR_ARG;
  if (int64_t(heads_q) + hk > 65536) return PRISM_ERR_UNSUPPORTED;
  if (n_tokens > 0 && (!q || !q_out)) return PRISM_ERR_ARG;
  if (!k != !k_out) return PRISM_ERR_ARG;
  const size_t es = dtype == PRISM_FP32 ? 4 : 2;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.src[0] = q; a.src[1] = k;
  a.dst[0] = q_out; a.dst[1] = k_out;
  a.src_ld[0] = q_stride; a.src_ld[1] = k_stride;
  a.dst_ld[0] = q_out_stride; a.dst_ld[1] = k_out_stride;
  const int tensors = k ? 2 : 1;
  uintptr_t bits = 0;  // of every address and byte stride
  bool in_place = true;
  for (int w = 0; w < tensors; ++w) {
    const int64_t width = int64_t(w ? heads_k : heads_q) * head_dim;
    if (a.src_ld[w] < width || a.dst_ld[w] < width) return PRISM_ERR_ARG;
    if (a.src_ld[w] > (int64_t(1) << 31) || a.dst_ld[w] > (int64_t(1) << 31)) return PRISM_ERR_UNSUPPORTED;
    bits |= reinterpret_cast<uintptr_t>(a.src[w]) | reinterpret_cast<uintptr_t>(a.dst[w]);
    bits |= uintptr_t(a.src_ld[w]) * es | uintptr_t(a.dst_ld[w]) * es;
    in_place = in_place && a.src[w] == a.dst[w] && a.src_ld[w] == a.dst_ld[w];
  }
  if (bits % es) return PRISM_ERR_ARG;
  if (n_tokens == 0) return PRISM_OK;
  // an output may be its own input; it may not meet the other tensors
  for (int w = 0; w < tensors; ++w)
    for (int v = 0; v < tensors; ++v) {
      const int64_t ww = int64_t(w ? heads_k : heads_q) * head_dim * es, wv = int64_t(v ? heads_k : heads_q) * head_dim * es;
      const uintptr_t d = reinterpret_cast<uintptr_t>(a.dst[w]);
      const bool own = v == w && a.src[w] == a.dst[w] && a.src_ld[w] == a.dst_ld[w];
      if (!own && rows_meet(d, a.dst_ld[w] * es, ww, reinterpret_cast<uintptr_t>(a.src[v]), a.src_ld[v] * es, wv, n_tokens))
        return PRISM_ERR_ARG;
      if (v > w && rows_meet(d, a.dst_ld[w] * es, ww, reinterpret_cast<uintptr_t>(a.dst[v]), a.dst_ld[v] * es, wv, n_tokens))
        return PRISM_ERR_ARG;
    }
  a.n = n_tokens;
  a.pos = positions;
  a.heads_q = heads_q;
  a.heads = heads_q + hk;
  a.head_dim = head_dim;
  a.pairs = rot / 2;
  a.axes = params->n_axes;
  a.pair1 = params->axis_dim[0] / 2;
  a.pair2 = a.axes == 3 ? a.pair1 + params->axis_dim[1] / 2 : a.pairs;
  a.grid_h = grid ? grid->h : 1;
  a.grid_w = grid ? grid->w : 1;
  a.m = float(params->magnitude);
  a.sign = transposed ? -1.f : 1.f;
  for (int x = 0, i = 0; x < a.axes; ++x)
    for (int j = 0; j < params->axis_dim[x] / 2; ++j, ++i) {
      const double f = pair_turns(*params, params->axis_dim[x], j);
      a.turn[i] = params->pos_scale[x] * f;
      a.start[i] = params->pos_offset[x] * f;
    }
  // the widest vector that divides the head, the half and every address and stride
  const bool half = params->layout == PRISM_ROPE_HALF;
  int ev = 16 / int(es);
  if (half) {
    while (ev > 1 && ((rot / 2) % ev || head_dim % ev || bits % (ev * es))) ev /= 2;
    a.rot_units = rot / 2 / ev;
    a.units = a.rot_units + (in_place ? 0 : (head_dim - rot) / ev);
  } else {
    if (head_dim % ev || bits % 16) ev = 2;
    a.rot_units = (rot + ev - 1) / ev;
    a.units = in_place ? a.rot_units : head_dim / ev;
  }
  // a CTA: `units` threads per head, as many heads as fit, then tokens side by side
  a.head_groups = kRopeThreads / a.units < a.heads ? kRopeThreads / a.units : a.heads;
  a.token_groups = kRopeThreads / (a.units * a.head_groups);
  // few tokens: a CTA each, for as many SMs as possible
  int64_t tok = n_tokens / (int64_t(device_sm_count()) * 8);
  if (tok > kRopeMaxTokens / 2) tok = kRopeMaxTokens / 2;
  if (tok < 1) tok = 1;
  if (a.token_groups > kRopeMaxTokens) a.token_groups = kRopeMaxTokens;
  if (a.token_groups > tok) {
    if (tok == 1) a.token_groups = 1;
    else tok = a.token_groups;
  }
  a.tokens = int(tok);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(dtype == PRISM_BF16 ? dispatch<__nv_bfloat16>(a, ev, half, s) : dispatch<float>(a, ev, half, s));
}
