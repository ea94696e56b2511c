// Rotary positions of Q and K, in the place where the block pooling, the
// scoring and the attention read them, and the transposed rotation of dQ and
// dK after the attention's backward pass.
//
// The mathematics. Pair i of a head (channels 2i, 2i + 1 interleaved, or i,
// i + rot/2 in halves) of the token at position p turns by the angle
//   a = (offset_x + p_x * scale_x) * f_i
// of its axis x (t, h, w of the token grid, or one given position):
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a).
// The transposed rotation (the gradient) is the same with -a. Only the
// fraction of a turn matters, so a / 2 pi is formed modulo 1 as a 64-bit fixed
// point number: the host gives scale f / 2 pi and offset f / 2 pi as fractions
// of 2^64 (from fp64), the kernel multiplies the first by the position and
// adds the second with wrap-around, exact for every int32 position. Its top 32
// bits become fp32 (off by 2^-26 turns at most) for sin and cos.
//
// What bounds it: HBM, every element read once and written once, three
// operations each. The angles depend on (token, pair) alone, so a CTA computes
// those of its few tokens once into shared memory and every head of Q and K
// reads them from there. A thread keeps one vector's place inside the head and
// walks the heads, so its cosines and sines sit in registers per token. All of
// a CTA's vectors are copied to shared memory asynchronously before the angles
// are computed (each thread reads back what it copied itself): 24 KB in flight
// per CTA and no registers held, where loads into registers left the kernel
// waiting on them. Q and K of the 2K grid (7.25 GB moved): 1.04 ms, 6.97 TB/s
// (the register version: 1.18 ms; flattening heads and tokens into one list of
// work cost 1.8 ms in index arithmetic).
//
// The half layout with a half that is no multiple of 16 bytes goes through
// rope_staged_kernel: whole rows in 16-byte vectors to shared memory, rotated
// there in place by narrower vectors, and back in 16-byte vectors.
//
// With one or two heads the angles are most of the work and the kernel is bound
// by instructions (2.6 times the floor for one head each of Q and K, 101 pairs; on a
// grid the angles of t and h are formed for each token, though its neighbours' are alike);
// the hardware's approximate sine and cosine would take 8 % off that and lose
// three bits, so the exact ones stay.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"

namespace prism {
namespace {

constexpr int kRopeMaxHeadDim = 256;
constexpr int kRopeMaxPairs = kRopeMaxHeadDim / 2;
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;       // of a CTA
constexpr int kRopeSmem = 24 * 1024;     // a CTA's vectors in flight
constexpr int kRopeMaxHeadGroups = 12;   // heads side by side: several heads per thread share its cosines and sines


// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery,
// "Division by invariant integers using multiplication").
struct FastDiv {
  uint32_t d, mul, shift;
};
FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  return {d, uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1), l};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const FastDiv& f) {
  return uint32_t((uint64_t(__umulhi(n, f.mul)) + n) >> f.shift);
}

struct RopeArgs {
  const void* src[2];  // Q, K
  void* dst[2];
  int64_t src_ld[2], dst_ld[2];  // elements between tokens
  int64_t n;                     // tokens
  const int32_t* pos;            // [n, axes], or null: the raster grid
  int heads[2];
  int head_dim, pairs;
  int axes;          // 1 or 3
  int pair1, pair2;  // first pair of axis 1, of axis 2
  FastDiv by_w, by_h, by_pairs;
  int rot_units, units;  // vectors (half: vector pairs) a head's rotated part has, and all that are touched
  int head_groups, token_groups, tokens;  // of a CTA
  int vec_offset;        // of the vectors in shared memory
  float m, sign;
  uint64_t turn[kRopeMaxPairs];   // turns per position, modulo 1, in 2^-64
  uint64_t start[kRopeMaxPairs];  // turns at position 0
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

// The rotated pair, its roundings spelt out: every variant gives the same bits.
__device__ __forceinline__ float turn1(float x1, float x2, float c, float s) { return fmaf(x1, c, -__fmul_rn(x2, s)); }
__device__ __forceinline__ float turn2(float x1, float x2, float c, float s) { return fmaf(x2, c, __fmul_rn(x1, s)); }

// BYTES (4, 8 or 16, aligned) from global to shared memory without a register.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}

// m cos a and m sin a (signed) of the CTA's tokens n0 .. n0 + end - 1, all pairs.
__device__ __forceinline__ void rope_angles(const RopeArgs& P, int64_t n0, int end, float* cosines, float* sines) {
  // Every lane wants another pair's entry: constant memory would serve one lane
  // at a time, so the tables are read as ordinary memory (the compiler cannot
  // see through the address any more).
  const uint64_t* turn = P.turn;
  const uint64_t* start = P.start;
  asm("" : "+l"(turn), "+l"(start));
  for (int x = threadIdx.x; x < end * P.pairs; x += blockDim.x) {
    const int tok = quotient(x, P.by_pairs), i = x - tok * P.pairs;
    const int64_t n = n0 + tok;
    const int axis = i < P.pair1 ? 0 : i < P.pair2 ? 1 : 2;
    int p = int(n);
    if (P.pos) {
      p = P.pos[n * P.axes + axis];
    } else if (P.axes == 3) {
      const uint32_t row = quotient(uint32_t(n), P.by_w), t = quotient(row, P.by_h);
      p = axis == 2 ? int(uint32_t(n) - row * P.by_w.d) : axis == 1 ? int(row - t * P.by_h.d) : int(t);
    }
    const uint64_t turns = uint64_t(int64_t(p)) * turn[i] + start[i];
    float s, c;
    sincospif(float(int32_t(turns >> 32)) * (1.f / 2147483648.f), &s, &c);
    cosines[x] = c * P.m;
    sines[x] = s * P.m * P.sign;
  }
}

// HALF: a unit is two vectors of EV elements, rot/2 apart; otherwise one
// vector of EV elements, EV/2 pairs. EV is the widest vector that the sizes,
// strides and addresses allow (16 bytes on every usual layout). With ELEM the
// vector's elements are loaded and stored one by one (an interleaved pair at
// an address that is no multiple of its size). MIXED: an interleaved vector
// may hold unrotated pairs; it is computed like the others, and they are kept.
template <typename T, int EV, bool HALF, bool ELEM, bool MIXED, bool ASYNC>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs P) {
  constexpr int kPairs = HALF ? EV : EV / 2;  // of a unit
  constexpr int kVecs = HALF ? 2 : 1;
  using V = Vec<T, EV>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const cosines = reinterpret_cast<float*>(smem);  // [tokens][pairs]: m cos a, then m sin a
  float* const sines = cosines + P.tokens * P.pairs;
  V* const mine = reinterpret_cast<V*>(smem + P.vec_offset) + threadIdx.x;  // every blockDim.x-th is this thread's
  const int64_t n0 = int64_t(blockIdx.x) * P.tokens;
  const int end = P.n - n0 < P.tokens ? int(P.n - n0) : P.tokens;
  const int group = threadIdx.x / P.units, u = threadIdx.x - group * P.units;
  const int tg = group / P.head_groups, hg = group - tg * P.head_groups;
  const bool rot = u < P.rot_units;
  // where the unit sits in the head, and its second vector (half layout) P.pairs further on
  const int c0 = HALF && !rot ? 2 * P.rot_units * EV + (u - P.rot_units) * EV : u * EV;
  const int step = P.head_groups * P.head_dim;
  if constexpr (ASYNC) {
    V* v = mine;
    for (int tok = tg; tok < end; tok += P.token_groups) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const T* x = static_cast<const T*>(P.src[w]) + (n0 + tok) * P.src_ld[w] + hg * P.head_dim + c0;
        for (int h = hg; h < P.heads[w]; h += P.head_groups, x += step, v += kVecs * blockDim.x) {
          copy_async<sizeof(V)>(v, x);
          if (HALF && rot) copy_async<sizeof(V)>(v + blockDim.x, x + P.pairs);
        }
      }
    }
  }
  rope_angles(P, n0, end, cosines, sines);
  if constexpr (ASYNC) asm volatile("cp.async.wait_all;" ::: "memory");  // this thread's own copies
  __syncthreads();
  const int valid = MIXED ? min(kPairs, P.pairs - u * kPairs) : kPairs;
  const V* v = mine;
  for (int tok = tg; tok < end; tok += P.token_groups) {
    float co[kPairs], si[kPairs];
    const int at = tok * P.pairs + u * kPairs;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const bool in = HALF ? rot : !MIXED || i < valid;
      co[i] = in ? cosines[at + i] : 0.f;
      si[i] = in ? sines[at + i] : 0.f;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const T* x = static_cast<const T*>(P.src[w]) + (n0 + tok) * P.src_ld[w] + hg * P.head_dim + c0;
      T* y = static_cast<T*>(P.dst[w]) + (n0 + tok) * P.dst_ld[w] + hg * P.head_dim + c0;
#pragma unroll 2
      for (int h = hg; h < P.heads[w]; h += P.head_groups, x += step, y += step) {
        V A, B;
        if constexpr (ASYNC) {
          A = v[0];
          if (HALF && rot) B = v[blockDim.x];
          v += kVecs * blockDim.x;
        } else if constexpr (ELEM) {
#pragma unroll
          for (int e = 0; e < EV; ++e) A.e[e] = x[e];
        } else {
          A = *reinterpret_cast<const V*>(x);
          if (HALF && rot) B = *reinterpret_cast<const V*>(x + P.pairs);
        }
        if constexpr (HALF) {
          if (rot) {
#pragma unroll
            for (int e = 0; e < EV; ++e) {
              const float x1 = to_f(A.e[e]), x2 = to_f(B.e[e]);
              A.e[e] = from_f<T>(turn1(x1, x2, co[e], si[e]));
              B.e[e] = from_f<T>(turn2(x1, x2, co[e], si[e]));
            }
            *reinterpret_cast<V*>(y + P.pairs) = B;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float x1 = to_f(A.e[2 * e]), x2 = to_f(A.e[2 * e + 1]);
            const T y1 = from_f<T>(turn1(x1, x2, co[e], si[e])), y2 = from_f<T>(turn2(x1, x2, co[e], si[e]));
            if (!MIXED || e < valid) {  // the others keep their bits, NaN and infinities too
              A.e[2 * e] = y1;
              A.e[2 * e + 1] = y2;
            }
          }
        }
        if constexpr (ELEM) {
#pragma unroll
          for (int e = 0; e < EV; ++e) y[e] = A.e[e];
        } else {
          *reinterpret_cast<V*>(y) = A;
        }
      }
    }
  }
}

// Half layout, rot / 2 any number of elements: 16-byte global accesses of whole
// rows (addresses, strides and row widths are multiples of 16 bytes), pairs of
// EV elements rotated in shared memory. `units` threads per head are the
// rotated ones alone; the other channels pass through with their row.
template <typename T, int EV>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_staged_kernel(const __grid_constant__ RopeArgs P) {
  using V = Vec<T, EV>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const cosines = reinterpret_cast<float*>(smem);
  float* const sines = cosines + P.tokens * P.pairs;
  T* const rows = reinterpret_cast<T*>(smem + P.vec_offset);  // [tokens][heads of Q, heads of K][head_dim]
  const int heads = P.heads[0] + P.heads[1], width = heads * P.head_dim;
  const int64_t n0 = int64_t(blockIdx.x) * P.tokens;
  const int end = P.n - n0 < P.tokens ? int(P.n - n0) : P.tokens;
  constexpr int kE = 16 / sizeof(T);
  const int vecs[2] = {P.heads[0] * P.head_dim / kE, P.heads[1] * P.head_dim / kE};
  for (int tok = 0; tok < end; ++tok)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const T* x = static_cast<const T*>(P.src[w]) + (n0 + tok) * P.src_ld[w];
      T* r = rows + tok * width + (w ? P.heads[0] * P.head_dim : 0);
      for (int i = threadIdx.x; i < vecs[w]; i += blockDim.x) copy_async<16>(r + i * kE, x + i * kE);
    }
  rope_angles(P, n0, end, cosines, sines);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int group = threadIdx.x / P.units, u = threadIdx.x - group * P.units;
  const int tg = group / P.head_groups, hg = group - tg * P.head_groups;
  for (int tok = tg; tok < end; tok += P.token_groups) {
    float co[EV], si[EV];
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      co[i] = cosines[tok * P.pairs + u * EV + i];
      si[i] = sines[tok * P.pairs + u * EV + i];
    }
    T* r = rows + tok * width + hg * P.head_dim + u * EV;
#pragma unroll 2
    for (int h = hg; h < heads; h += P.head_groups, r += P.head_groups * P.head_dim) {
      V A = *reinterpret_cast<const V*>(r), B = *reinterpret_cast<const V*>(r + P.pairs);
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const float x1 = to_f(A.e[e]), x2 = to_f(B.e[e]);
        A.e[e] = from_f<T>(turn1(x1, x2, co[e], si[e]));
        B.e[e] = from_f<T>(turn2(x1, x2, co[e], si[e]));
      }
      *reinterpret_cast<V*>(r) = A;
      *reinterpret_cast<V*>(r + P.pairs) = B;
    }
  }
  __syncthreads();
  for (int tok = 0; tok < end; ++tok)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      T* y = static_cast<T*>(P.dst[w]) + (n0 + tok) * P.dst_ld[w];
      const T* r = rows + tok * width + (w ? P.heads[0] * P.head_dim : 0);
      for (int i = threadIdx.x; i < vecs[w]; i += blockDim.x)
        *reinterpret_cast<uint4*>(y + i * kE) = *reinterpret_cast<const uint4*>(r + i * kE);
    }
}

// Turns per position of the pairs of an axis with n rotated channels. The
// powers theta^(-2j/n) come one from the other in extended precision, exact to
// fp64 for every j.
void axis_turns(const prism_rope_params& r, int n, double* turns) {
  const long double two_pi = 6.283185307179586476925286766559L;
  double theta = r.theta;
  if (r.scaling == PRISM_ROPE_NTK && n > 2) theta *= std::pow(r.factor, double(n) / (n - 2));
  // with YaRN, pairs that turn more than 32 times over the trained length keep their frequency, those below one turn
  // are stretched, a ramp over the index between
  double low = 0.0, width = 1.0;
  if (r.scaling == PRISM_ROPE_YARN) {
    const double per = n / (2.0 * std::log(theta));
    low = std::fmax(std::floor(per * std::log(r.trained_len / (32.0 * double(two_pi)))), 0.0);
    const double high = std::fmin(std::ceil(per * std::log(r.trained_len / double(two_pi))), double(n - 1));
    width = std::fmax(high - low, 0.001);
  }
  const long double step = powl(theta, -2.0L / n);
  long double f = 1.0L / two_pi;
  for (int j = 0; j < n / 2; ++j, f *= step) {
    double share = r.scaling == PRISM_ROPE_LINEAR ? 1.0 : 0.0;  // of the stretched frequency
    if (r.scaling == PRISM_ROPE_YARN) share = std::fmin(std::fmax((j - low) / width, 0.0), 1.0);
    turns[j] = share == 0.0 ? double(f) : double(f) / r.factor * share + double(f) * (1.0 - share);
  }
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

// Shared memory of a CTA's vectors.
int rope_vec_bytes(const RopeArgs& a, int vec, bool half) {
  const int per_token = (a.heads[0] + a.head_groups - 1) / a.head_groups + (a.heads[1] + a.head_groups - 1) / a.head_groups;
  const int tokens = (a.tokens + a.token_groups - 1) / a.token_groups;
  return tokens * per_token * (half ? 2 : 1) * a.units * a.head_groups * a.token_groups * vec;
}

template <typename T, int EV, bool HALF, bool ELEM, bool MIXED, bool ASYNC>
cudaError_t launch_as(const RopeArgs& a, int smem, cudaStream_t s) {
  const int64_t ctas = (a.n + a.tokens - 1) / a.tokens;
  const int threads = a.units * a.head_groups * a.token_groups;
  auto kernel = rope_kernel<T, EV, HALF, ELEM, MIXED, ASYNC>;
  kernel<<<unsigned(ctas), threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int EV, bool HALF, bool ELEM, bool MIXED>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int vec = EV * int(sizeof(T)), bytes = rope_vec_bytes(a, vec, HALF);
  if constexpr (!ELEM && EV * sizeof(T) >= 4) {
    if (bytes <= kRopeSmem) return launch_as<T, EV, HALF, ELEM, MIXED, true>(a, a.vec_offset + bytes, s);
  }
  return launch_as<T, EV, HALF, ELEM, MIXED, false>(a, a.vec_offset, s);
}
template <typename T>
cudaError_t dispatch(const RopeArgs& a, int ev, bool half, cudaStream_t s) {
  constexpr int kWide = 16 / int(sizeof(T));
  if (!half) {
    if (ev != kWide) return launch<T, 2, false, true, true>(a, s);
    if (a.pairs < a.units * (kWide / 2)) return launch<T, kWide, false, false, true>(a, s);
    return launch<T, kWide, false, false, false>(a, s);
  }
  if constexpr (kWide == 8) {
    if (ev == 8) return launch<T, 8, true, false, false>(a, s);
  }
  if (ev == 4) return launch<T, 4, true, false, false>(a, s);
  if (ev == 2) return launch<T, 2, true, false, false>(a, s);
  return launch<T, 1, true, false, false>(a, s);
}

template <typename T, int EV>
cudaError_t launch_staged(const RopeArgs& a, int smem, cudaStream_t s) {
  const int64_t ctas = (a.n + a.tokens - 1) / a.tokens;
  rope_staged_kernel<T, EV><<<unsigned(ctas), a.units * a.head_groups * a.token_groups, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch_staged(const RopeArgs& a, int ev, int smem, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (ev == 4) return launch_staged<T, 4>(a, smem, s);
  }
  return ev == 2 ? launch_staged<T, 2>(a, smem, s) : launch_staged<T, 1>(a, smem, s);
}

// x modulo 1 in units of 2^-64 (its two's complement for a negative x).
uint64_t fraction_bits(double x) {
  if (x == 0.0) return 0;
  const double r = std::fabs(x) < 1.0 ? x : std::fmod(x, 1.0);  // exact
  const uint64_t b = uint64_t(std::fabs(r) * 18446744073709551616.0);
  return r < 0.0 ? uint64_t(0) - b : b;
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
      if (positions && rows_meet(d, a.dst_ld[w] * es, ww, reinterpret_cast<uintptr_t>(positions),
                                 int64_t(params->n_axes) * 4, int64_t(params->n_axes) * 4, n_tokens))
        return PRISM_ERR_ARG;
    }
  a.n = n_tokens;
  a.pos = positions;
  a.heads[0] = heads_q;
  a.heads[1] = hk;
  a.head_dim = head_dim;
  a.pairs = rot / 2;
  a.axes = params->n_axes;
  a.pair1 = params->axis_dim[0] / 2;
  a.pair2 = a.axes == 3 ? a.pair1 + params->axis_dim[1] / 2 : a.pairs;
  const bool raster = a.axes == 3 && !positions;
  a.by_h = fast_div(raster ? grid->h : 1);
  a.by_w = fast_div(raster ? grid->w : 1);
  a.by_pairs = fast_div(a.pairs);
  a.m = float(params->magnitude);
  a.sign = transposed ? -1.f : 1.f;
  double turns[kRopeMaxPairs];
  for (int x = 0, i = 0; x < a.axes; ++x) {
    if (params->axis_dim[x] == 0) continue;
    axis_turns(*params, params->axis_dim[x], turns);
    for (int j = 0; j < params->axis_dim[x] / 2; ++j, ++i) {
      a.turn[i] = fraction_bits(params->pos_scale[x] * turns[j]);
      a.start[i] = fraction_bits(params->pos_offset[x] * turns[j]);
    }
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
  // a CTA: `units` threads per head, the heads of Q and of K in equal steps, then tokens side by side
  const int fit = kRopeThreads / a.units < kRopeMaxHeadGroups ? kRopeThreads / a.units : kRopeMaxHeadGroups;
  a.head_groups = 1;
  for (int g = 2; g <= fit; ++g) {  // the most heads side by side that leave at most a tenth of the places idle
    const int64_t places = (int64_t(heads_q + g - 1) / g + (hk + g - 1) / g) * g;
    if (places * 10 <= int64_t(heads_q + hk) * 11) a.head_groups = g;
  }
  a.token_groups = kRopeThreads / (a.units * a.head_groups);
  // tokens of a CTA: its vectors fill kRopeSmem; few tokens: fewer, for as many SMs as possible
  int64_t tok = n_tokens / (int64_t(device_sm_count()) * 2);
  if (tok < 1) tok = 1;
  if (tok > kRopeMaxTokens) tok = kRopeMaxTokens;
  if (a.token_groups > tok) a.token_groups = int(tok);
  a.tokens = a.token_groups;
  const int vec = ev * int(es);
  while (a.tokens + a.token_groups <= tok) {
    a.tokens += a.token_groups;
    if (rope_vec_bytes(a, vec, half) > kRopeSmem) {
      a.tokens -= a.token_groups;
      break;
    }
  }
  while (a.token_groups > 1 && rope_vec_bytes(a, vec, half) > kRopeSmem) a.tokens = --a.token_groups;
  // a half of no whole vectors, rows of whole vectors: through shared memory
  const int64_t row = int64_t(heads_q + hk) * head_dim * es;
  const bool staged = half && vec < 16 && bits % 16 == 0 && (int64_t(heads_q) * head_dim * es) % 16 == 0 &&
                      (int64_t(hk) * head_dim * es) % 16 == 0 && row <= kRopeSmem;
  if (staged) {
    a.units = a.rot_units;
    a.head_groups = std::min(std::min(kRopeThreads / a.units, heads_q + hk), kRopeMaxHeadGroups);
    a.token_groups = int(std::min<int64_t>(kRopeThreads / (a.units * a.head_groups), tok));
    a.tokens = int(std::min<int64_t>(tok, kRopeSmem / row));
    if (a.token_groups > a.tokens) a.token_groups = a.tokens;
  }
  a.vec_offset = (a.tokens * a.pairs * 8 + 15) / 16 * 16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (staged) {
    const int smem = a.vec_offset + a.tokens * int(row);
    return cuda_status(dtype == PRISM_BF16 ? dispatch_staged<__nv_bfloat16>(a, ev, smem, s)
                                           : dispatch_staged<float>(a, ev, smem, s));
  }
  return cuda_status(dtype == PRISM_BF16 ? dispatch<__nv_bfloat16>(a, ev, half, s) : dispatch<float>(a, ev, half, s));
}
