// The global norm of a list of gradients, and their clipping by it: what ends
// the backward pass of a training step.
//
// The mathematics. norm = sqrt(sum over every element of every tensor of g^2)
// (or the largest |g|), and then g <- g * min(1, max_norm / (norm + eps)).
//
// Sums. A thread squares and adds the elements of a few 16-byte vectors in
// fp32 (kVecs vectors: at most 32 terms in two chains), and adds that to an
// fp64 sum; a group whose fp32 sum overflowed, or is so small that its squares
// may have lost bits below the smallest normal number, is squared again in
// fp64, so gradients of any magnitude that their type holds count in full. The
// CTAs' sums are written to the workspace and added in a fixed order: no
// atomics, the same result every time.
//
// Work. The tensors are cut into chunks of 16 KB, which the CTAs take in turn;
// the next chunk is loaded while one is worked on. The table of tensors travels
// as a kernel parameter (kMany entries per launch), so nothing is copied to the
// device and a captured graph carries its own table.
//
// What bounds it: HBM. The norm reads every element once; the scaling reads and
// writes each once more, which it has to, since no element may be written
// before the last one has been read. The scaling pass walks the chunks
// backwards, so that what the norm pass read last (up to the size of L2) is
// found there. 600 M bf16 values in 64 tensors: norm 0.19 ms (6.3 TB/s), with the
// scaling 0.59 ms (3.6 GB moved; without the loads ahead 0.63; 3 to 8 CTAs per SM
// and 2 to 8 vectors measured: 4 of each is within 2 % of the best on large lists,
// more CTAs spill registers or crowd the memory system).
//
// Small lists (at most kSmallChunks chunks) take one launch: a cluster of CTAs
// reads every value once into registers, the sums meet in distributed shared
// memory, and the values are scaled from the registers. 40,001 fp32 values in 6
// tensors: 4.7 us on the GPU like the two launches, and 2 us less of the host (10.3 for
// the whole Python call, 12.3).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "host.h"

namespace prism {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnVecs = 4;                                // 16-byte vectors of a thread per chunk
constexpr int kGnChunkVecs = kGnThreads * kGnVecs;        // 16 KB
constexpr int kGnCtasPerSm = 4;
constexpr int kGnMaxCtas = 148 * kGnCtasPerSm;
constexpr int kMany = 900, kFew = 40;                     // tensors per launch (a kernel takes 32,764 bytes of parameters)

struct GnItem {
  const char* src;
  char* dst;
  int64_t n;       // elements
  int32_t chunk0;  // first chunk of the launch that is this tensor's
  int32_t fp32;
};

template <int CAP>
struct GnTable {
  int32_t items, chunks;
  int32_t inf_norm;
  GnItem item[CAP];
};

__device__ __forceinline__ bool tiny_or_over(float s) { return !(s > 1e-30f && s < 3e38f); }

// Where this thread's vectors of a chunk lie: `at` the address of the first,
// rounded down to 16, the tensor's bytes being [lo, hi).
struct GnPlace {
  uintptr_t at, lo, hi;
  intptr_t delta;  // from a value to where it goes
  bool fp32;
};
template <int CAP>
__device__ __forceinline__ GnPlace place(const GnTable<CAP>& T, int chunk, int item) {
  const GnItem& I = T.item[item];
  GnPlace p;
  p.lo = reinterpret_cast<uintptr_t>(I.src);
  p.hi = p.lo + uintptr_t(I.n) * (I.fp32 ? 4 : 2);
  p.at = (p.lo & ~uintptr_t(15)) + (uintptr_t(chunk - I.chunk0) * kGnChunkVecs + threadIdx.x) * 16;
  p.delta = I.dst - I.src;
  p.fp32 = I.fp32;
  return p;
}

// Values outside the tensor count as zero.
__device__ __forceinline__ void load_chunk(const GnPlace& p, uint4* v) {
#pragma unroll
  for (int i = 0; i < kGnVecs; ++i) {
    const uintptr_t a = p.at + uintptr_t(i) * kGnThreads * 16;
    if (a >= p.lo && a + 16 <= p.hi) {
      v[i] = *reinterpret_cast<const uint4*>(a);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
      if (a < p.hi) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uintptr_t q = a + 2 * e;
          if (q >= p.lo && q < p.hi) w[e >> 1] |= uint32_t(*reinterpret_cast<const uint16_t*>(q)) << ((e & 1) * 16);
        }
      }
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <bool FP32>
struct Chunk {
  static constexpr int kE = FP32 ? 4 : 8;
  const uint4* v;

  static __device__ __forceinline__ void decode(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FP32) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  __device__ __forceinline__ double sum_squares() const {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kGnVecs; ++i) {
      float x[kE];
      decode(v[i], x);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        s0 = fmaf(x[e], x[e], s0);
        s1 = fmaf(x[e + 1], x[e + 1], s1);
      }
    }
    const float s = s0 + s1;
    if (!tiny_or_over(s)) return double(s);
    if (s == 0.f && max_bits() == 0) return 0.0;  // gradients that are all zero, not just small
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < kGnVecs; ++i) {
      float x[kE];
      decode(v[i], x);
#pragma unroll
      for (int e = 0; e < kE; ++e) d = fma(double(x[e]), double(x[e]), d);
    }
    return d;
  }
  // The bits of the largest magnitude: their order is the values', NaN above infinity.
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kGnVecs; ++i) {
      float x[kE];
      decode(v[i], x);
#pragma unroll
      for (int e = 0; e < kE; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    }
    return m;
  }
  // The values times f, rounded once, to p.delta bytes further on; whole
  // vectors where both sides are aligned.
  __device__ __forceinline__ void store_scaled(float f, const GnPlace& p) const {
#pragma unroll
    for (int i = 0; i < kGnVecs; ++i) {
      const uintptr_t a = p.at + uintptr_t(i) * kGnThreads * 16;
      if (a >= p.hi) continue;
      float x[kE];
      decode(v[i], x);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (FP32) {
          w[j] = __float_as_uint(x[j] * f);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j] * f, x[2 * j + 1] * f);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if (a >= p.lo && a + 16 <= p.hi && p.delta % 16 == 0) {
        *reinterpret_cast<uint4*>(a + p.delta) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uintptr_t q = a + 2 * e;
          if (q >= p.lo && q < p.hi) *reinterpret_cast<uint16_t*>(q + p.delta) = uint16_t(w[e >> 1] >> ((e & 1) * 16));
        }
      }
    }
  }
};

template <int CAP>
__device__ __forceinline__ int find_item(const GnTable<CAP>& T, int chunk, int lo, int hi) {
  // the last item of lo .. hi whose first chunk is not behind `chunk`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (T.item[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Deterministic sum (or maximum) over the CTA; the result is thread 0's.
__device__ __forceinline__ double cta_reduce(double d, bool maximum) {
  __shared__ double part[kGnThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const double x = __shfl_down_sync(0xffffffffu, d, o);
    d = maximum ? (x > d ? x : d) : d + x;
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kGnThreads / 32; ++i) d = maximum ? (part[i] > d ? part[i] : d) : d + part[i];
  return d;
}

// Pass 1: CTA b's chunks, every gridDim.x-th from b on, to partial[b]: a sum of squares, or the largest magnitude's bits as a number.
template <int CAP>
__global__ void __launch_bounds__(kGnThreads, kGnCtasPerSm) norm_kernel(const __grid_constant__ GnTable<CAP> T, double* partial) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int c = blockIdx.x;
  double acc = 0.0;
  uint32_t top = 0;
  {
    int it = find_item(T, c, 0, T.items - 1);
    GnPlace p = place(T, c, it);
    uint4 v[kGnVecs];
    load_chunk(p, v);
    while (true) {
      // the next chunk is on its way while this one is added
      GnPlace pn = p;
      uint4 vn[kGnVecs];
      c += gridDim.x;
      const bool more = c < T.chunks;
      if (more) {
        if (it + 1 < T.items && T.item[it + 1].chunk0 <= c) it = find_item(T, c, it + 1, T.items - 1);
        pn = place(T, c, it);
        load_chunk(pn, vn);
      }
      if (p.fp32) {
        const Chunk<true> k{v};
        if (T.inf_norm) top = max(top, k.max_bits());
        else acc += k.sum_squares();
      } else {
        const Chunk<false> k{v};
        if (T.inf_norm) top = max(top, k.max_bits());
        else acc += k.sum_squares();
      }
      if (!more) break;
      p = pn;
#pragma unroll
      for (int i = 0; i < kGnVecs; ++i) v[i] = vn[i];
    }
  }
  const double r = cta_reduce(T.inf_norm ? double(top) : acc, T.inf_norm);
  if (threadIdx.x == 0) partial[blockIdx.x] = r;
}

// The norm from every CTA's part, in a fixed order, to every thread of the CTA.
__device__ __forceinline__ double combine(const double* partial, int parts, bool inf_norm) {
  __shared__ double norm;
  double d = 0.0;
  for (int i = threadIdx.x; i < parts; i += kGnThreads) {
    const double x = partial[i];
    d = inf_norm ? (x > d ? x : d) : d + x;
  }
  d = cta_reduce(d, inf_norm);
  if (threadIdx.x == 0) norm = inf_norm ? double(__uint_as_float(uint32_t(d))) : sqrt(d);
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(kGnThreads) finish_kernel(const double* partial, int parts, int inf_norm, float* norm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const double r = combine(partial, parts, inf_norm);
  if (threadIdx.x == 0) *norm = float(r);
}

struct GnScale {
  const double* partial;  // null: the norm is read from `norm`
  int32_t parts, inf_norm;
  float* norm;
  int32_t write_norm;
  float max_norm, eps;
};

// A NaN norm makes every value NaN, unless there is nothing to clip to; a norm
// of 0 (and eps = 0) leaves the values, with a bound of 0 too.
__device__ __forceinline__ float clip_factor(const GnScale& S, double norm) {
  const double by = norm + double(S.eps), f = double(S.max_norm) / by;
  return f >= 1.0 || by == 0.0 || isinf(S.max_norm) ? 1.f : float(f);
}

// Pass 2: the factor, and this CTA's chunks times it, last chunk first.
template <int CAP>
__global__ void __launch_bounds__(kGnThreads, kGnCtasPerSm) scale_kernel(const __grid_constant__ GnTable<CAP> T, const GnScale S) {
  const int step = int(gridDim.x);
  int c = int(blockIdx.x) + (T.chunks - 1 - int(blockIdx.x)) / step * step;
  int it = find_item(T, c, 0, T.items - 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the norm pass, where this launch was let in beside its end
  const double norm = S.partial ? combine(S.partial, S.parts, S.inf_norm) : double(*S.norm);
  if (S.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *S.norm = float(norm);
  const float factor = clip_factor(S, norm);
  auto skip = [&](int c) {  // nothing to do for chunk c; also finds its item
    if (T.item[it].chunk0 > c) it = find_item(T, c, 0, it - 1);
    return factor == 1.f && T.item[it].src == T.item[it].dst;
  };
  while (c >= 0 && skip(c)) c -= step;
  if (c < 0) return;
  GnPlace p = place(T, c, it);
  uint4 v[kGnVecs];
  load_chunk(p, v);
  while (true) {
    GnPlace pn = p;
    uint4 vn[kGnVecs];
    c -= step;
    while (c >= 0 && skip(c)) c -= step;
    const bool more = c >= 0;
    if (more) {
      pn = place(T, c, it);
      load_chunk(pn, vn);
    }
    if (p.fp32) Chunk<true>{v}.store_scaled(factor, p);
    else Chunk<false>{v}.store_scaled(factor, p);
    if (!more) break;
    p = pn;
#pragma unroll
    for (int i = 0; i < kGnVecs; ++i) v[i] = vn[i];
  }
}

// Launches a kernel behind the norm pass of the same call, set up beside its end.
template <typename... K, typename... A>
cudaError_t launch_behind(void (*kernel)(K...), int ctas, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kGnThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The whole of a small list in one launch of one cluster: chunk c is CTA c mod
// kSmallCtas's; with `scale` the values are scaled, else only the norm is
// written. The order of the sums is the chunks' and the ranks': fixed.
constexpr int kSmallCtas = 8, kSmallPer = 4, kSmallChunks = kSmallCtas * kSmallPer;

__global__ void __cluster_dims__(kSmallCtas) __launch_bounds__(kGnThreads)
    small_kernel(const __grid_constant__ GnTable<kFew> T, const GnScale S, const int scale) {
  __shared__ double part;
  GnPlace p[kSmallPer];
  uint4 v[kSmallPer][kGnVecs];
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i) {
    const int c = int(blockIdx.x) + i * kSmallCtas;
    if (c < T.chunks) {
      p[i] = place(T, c, find_item(T, c, 0, T.items - 1));
      load_chunk(p[i], v[i]);
    }
  }
  double acc = 0.0;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i)
    if (int(blockIdx.x) + i * kSmallCtas < T.chunks) {
      if (T.inf_norm) top = max(top, p[i].fp32 ? Chunk<true>{v[i]}.max_bits() : Chunk<false>{v[i]}.max_bits());
      else acc += p[i].fp32 ? Chunk<true>{v[i]}.sum_squares() : Chunk<false>{v[i]}.sum_squares();
    }
  const double mine = cta_reduce(T.inf_norm ? double(top) : acc, T.inf_norm);
  if (threadIdx.x == 0) part = mine;
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  double norm = 0.0;
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&part));
#pragma unroll
  for (int r = 0; r < kSmallCtas; ++r) {
    double x;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f64 %0, [a];\n\t}"
        : "=d"(x)
        : "r"(at), "r"(r));
    norm = T.inf_norm ? (x > norm ? x : norm) : norm + x;
  }
  // every part is read before any CTA leaves
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  norm = T.inf_norm ? double(__uint_as_float(uint32_t(norm))) : sqrt(norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *S.norm = float(norm);
  if (scale) {
    const float factor = clip_factor(S, norm);
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i)
      if (int(blockIdx.x) + i * kSmallCtas < T.chunks && !(factor == 1.f && p[i].delta == 0)) {
        if (p[i].fp32) Chunk<true>{v[i]}.store_scaled(factor, p[i]);
        else Chunk<false>{v[i]}.store_scaled(factor, p[i]);
      }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

prism_status check_tensors(const prism_tensor* t, int64_t n, bool writes) {
  if (n < 0 || (n > 0 && !t)) return PRISM_ERR_ARG;
  if (n > (1 << 20)) return PRISM_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].numel < 0) return PRISM_ERR_ARG;
    if (t[i].dtype != PRISM_BF16 && t[i].dtype != PRISM_FP32) return PRISM_ERR_DTYPE;
    if (t[i].numel == 0) continue;
    const uintptr_t es = t[i].dtype == PRISM_FP32 ? 4 : 2;
    if (!t[i].data || reinterpret_cast<uintptr_t>(t[i].data) % es) return PRISM_ERR_ARG;
    if (writes && reinterpret_cast<uintptr_t>(t[i].out) % es) return PRISM_ERR_ARG;
    if (t[i].numel > (int64_t(1) << 43)) return PRISM_ERR_UNSUPPORTED;
  }
  return PRISM_OK;
}

// What one tensor's scaling writes may meet neither another tensor nor the norm
// nor, other than exactly, its own input.
prism_status check_apart(const prism_tensor* t, int64_t n, const float* norm) {
  struct Range {
    uintptr_t a, e;
    bool written;
  };
  try {
    std::vector<Range> r;
    r.reserve(size_t(n) * 2 + 1);
    r.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, false});
    for (int64_t i = 0; i < n; ++i) {
      if (!t[i].numel) continue;
      const uintptr_t bytes = uintptr_t(t[i].numel) * (t[i].dtype == PRISM_FP32 ? 4 : 2);
      const uintptr_t s = reinterpret_cast<uintptr_t>(t[i].data);
      const uintptr_t d = t[i].out ? reinterpret_cast<uintptr_t>(t[i].out) : s;
      r.push_back({d, d + bytes, true});
      if (d != s) r.push_back({s, s + bytes, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
    uintptr_t end = 0, end_written = 0;  // of the ranges so far
    for (const Range& x : r) {
      if (x.a < end_written || (x.written && x.a < end)) return PRISM_ERR_ARG;
      end = std::max(end, x.e);
      if (x.written) end_written = std::max(end_written, x.e);
    }
  } catch (...) {
    return PRISM_ERR_UNSUPPORTED;  // no host memory for the check
  }
  return PRISM_OK;
}

// The norm and the workspace are written: neither may meet the other or a
// gradient, nor the workspace a scaled one.
prism_status check_written(const prism_tensor* t, int64_t n, const float* norm, const void* ws, size_t bytes, bool scaled) {
  const uintptr_t m = reinterpret_cast<uintptr_t>(norm), w = reinterpret_cast<uintptr_t>(ws);
  auto over = [](uintptr_t a, uintptr_t na, uintptr_t b, uintptr_t nb) { return a < b + nb && b < a + na; };
  if (over(m, 4, w, bytes)) return PRISM_ERR_ARG;
  for (int64_t i = 0; i < n; ++i) {
    if (!t[i].numel) continue;
    const uintptr_t size = uintptr_t(t[i].numel) * (t[i].dtype == PRISM_FP32 ? 4 : 2);
    const uintptr_t s = reinterpret_cast<uintptr_t>(t[i].data), d = reinterpret_cast<uintptr_t>(t[i].out);
    if (over(s, size, w, bytes) || over(s, size, m, 4)) return PRISM_ERR_ARG;
    if (scaled && d && (over(d, size, w, bytes) || over(d, size, m, 4))) return PRISM_ERR_ARG;
  }
  return PRISM_OK;
}

int64_t chunks_of(const prism_tensor& t) {
  const int64_t bytes = t.numel * (t.dtype == PRISM_FP32 ? 4 : 2) + int64_t(reinterpret_cast<uintptr_t>(t.data) % 16);
  return (bytes + kGnChunkVecs * 16 - 1) / (kGnChunkVecs * 16);
}

// Launches of at most CAP tensors each; F(table, grid, first partial).
template <int CAP, typename F>
prism_status each_launch(const prism_tensor* t, int64_t n, bool inf_norm, const F& run) {
  GnTable<CAP> T;
  int64_t i = 0;
  int parts = 0;
  while (i < n) {
    T.items = 0;
    T.inf_norm = inf_norm;
    int64_t chunks = 0;
    for (; i < n && T.items < CAP; ++i) {
      if (!t[i].numel) continue;
      const int64_t c = chunks_of(t[i]);
      if (chunks + c > (int64_t(1) << 30)) {
        if (T.items == 0) return PRISM_ERR_UNSUPPORTED;
        break;
      }
      GnItem& I = T.item[T.items++];
      I.src = static_cast<const char*>(t[i].data);
      I.dst = static_cast<char*>(t[i].out ? t[i].out : t[i].data);
      I.n = t[i].numel;
      I.fp32 = t[i].dtype == PRISM_FP32;
      I.chunk0 = int32_t(chunks);
      chunks += c;
    }
    if (T.items == 0) break;
    T.chunks = int32_t(chunks);
    const int64_t ctas = std::min<int64_t>(chunks, std::min(device_sm_count() * kGnCtasPerSm, kGnMaxCtas));
    const cudaError_t e = run(T, int(ctas), parts);
    if (e != cudaSuccess) return PRISM_ERR_CUDA;
    parts += int(ctas);
  }
  return PRISM_OK;
}

// A small list in one launch; false when it is none.
bool run_small(const prism_tensor* t, int64_t n, const GnScale& g, int scale, cudaStream_t s, prism_status* st) {
  if (n > kFew) return false;
  int64_t chunks = 0;
  for (int64_t i = 0; i < n && chunks <= kSmallChunks; ++i)
    if (t[i].numel > kSmallChunks * kGnChunkVecs * 8) return false;
    else if (t[i].numel) chunks += chunks_of(t[i]);
  if (chunks == 0 || chunks > kSmallChunks) return false;
  *st = each_launch<kFew>(t, n, g.inf_norm, [&](const GnTable<kFew>& T, int, int) {
    small_kernel<<<kSmallCtas, kGnThreads, 0, s>>>(T, g, scale);
    return cudaGetLastError();
  });
  return true;
}

size_t norm_ws_bytes(int64_t n) {
  const int64_t launches = n / kMany + 2;
  return kWsHeader + align_up(size_t(launches) * kGnMaxCtas * sizeof(double), 256);
}

prism_status check_norm_ws(void* ws, size_t ws_bytes, int64_t n) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < norm_ws_bytes(n)) return PRISM_ERR_WORKSPACE;
  return PRISM_OK;
}

template <int CAP>
prism_status run_norm(const prism_tensor* t, int64_t n, bool inf_norm, double* partial, int* parts, cudaStream_t s) {
  return each_launch<CAP>(t, n, inf_norm, [&](const GnTable<CAP>& T, int ctas, int at) {
    norm_kernel<CAP><<<ctas, kGnThreads, 0, s>>>(T, partial + at);
    *parts = at + ctas;
    return cudaGetLastError();
  });
}

template <int CAP>
prism_status run_scale(const prism_tensor* t, int64_t n, GnScale g, cudaStream_t s) {
  return each_launch<CAP>(t, n, g.inf_norm, [&](const GnTable<CAP>& T, int ctas, int) {
    // the first launch follows the norm pass's last; prism_grad_scale's, and the later ones, run in plain order
    if (g.write_norm) {
      const cudaError_t e = launch_behind(scale_kernel<CAP>, ctas, s, T, g);
      g.write_norm = 0;
      return e;
    }
    scale_kernel<CAP><<<ctas, kGnThreads, 0, s>>>(T, g);
    return cudaGetLastError();
  });
}

prism_status norm_parts(const prism_tensor* t, int64_t n, int32_t ord, void* ws, double** partial, int* parts,
                        cudaStream_t s) {
  *partial = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kWsHeader);
  *parts = 0;
  const bool inf_norm = ord == PRISM_NORM_INF;
  return n <= kFew ? run_norm<kFew>(t, n, inf_norm, *partial, parts, s)
                   : run_norm<kMany>(t, n, inf_norm, *partial, parts, s);
}

bool bad_bound(float max_norm, float eps) { return !(max_norm >= 0.f) || !(eps >= 0.f) || std::isinf(eps); }

}  // namespace
}  // namespace prism

using namespace prism;

extern "C" prism_status prism_grad_norm_workspace_size(int64_t n_tensors, size_t* bytes) {
  if (!bytes || n_tensors < 0) return PRISM_ERR_ARG;
  if (n_tensors > (1 << 20)) return PRISM_ERR_UNSUPPORTED;
  *bytes = norm_ws_bytes(n_tensors);
  return PRISM_OK;
}

extern "C" prism_status prism_grad_norm(const prism_tensor* grads, int64_t n_tensors, int32_t ord, float* norm,
                                        void* ws, size_t ws_bytes, void* stream) {
  if (!norm || reinterpret_cast<uintptr_t>(norm) % 4) return PRISM_ERR_ARG;
  if (ord != PRISM_NORM_L2 && ord != PRISM_NORM_INF) return PRISM_ERR_ARG;
  prism_status st = check_tensors(grads, n_tensors, false);
  if (st == PRISM_OK) st = check_norm_ws(ws, ws_bytes, n_tensors);
  if (st == PRISM_OK) st = check_written(grads, n_tensors, norm, ws, norm_ws_bytes(n_tensors), false);
  if (st != PRISM_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const GnScale small = {nullptr, 0, ord == PRISM_NORM_INF, norm, 1, 0.f, 0.f};
  if (run_small(grads, n_tensors, small, 0, s, &st)) return st;
  double* partial;
  int parts;
  st = norm_parts(grads, n_tensors, ord, ws, &partial, &parts, s);
  if (st != PRISM_OK) return st;
  return cuda_status(launch_behind(finish_kernel, 1, s, partial, parts, int(ord == PRISM_NORM_INF), norm));
}

extern "C" prism_status prism_grad_scale(const prism_tensor* grads, int64_t n_tensors, const float* norm,
                                         float max_norm, float eps, void* stream) {
  if (!norm || reinterpret_cast<uintptr_t>(norm) % 4 || bad_bound(max_norm, eps)) return PRISM_ERR_ARG;
  prism_status st = check_tensors(grads, n_tensors, true);
  if (st == PRISM_OK) st = check_apart(grads, n_tensors, norm);
  if (st != PRISM_OK) return st;
  GnScale g = {nullptr, 0, 0, const_cast<float*>(norm), 0, max_norm, eps};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return n_tensors <= kFew ? run_scale<kFew>(grads, n_tensors, g, s) : run_scale<kMany>(grads, n_tensors, g, s);
}

extern "C" prism_status prism_grad_clip(const prism_tensor* grads, int64_t n_tensors, int32_t ord, float max_norm,
                                        float eps, float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (!norm || reinterpret_cast<uintptr_t>(norm) % 4 || bad_bound(max_norm, eps)) return PRISM_ERR_ARG;
  if (ord != PRISM_NORM_L2 && ord != PRISM_NORM_INF) return PRISM_ERR_ARG;
  prism_status st = check_tensors(grads, n_tensors, true);
  if (st == PRISM_OK) st = check_norm_ws(ws, ws_bytes, n_tensors);
  if (st == PRISM_OK) st = check_written(grads, n_tensors, norm, ws, norm_ws_bytes(n_tensors), true);
  if (st == PRISM_OK) st = check_apart(grads, n_tensors, norm);
  if (st != PRISM_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const GnScale small = {nullptr, 0, ord == PRISM_NORM_INF, norm, 1, max_norm, eps};
  if (run_small(grads, n_tensors, small, 1, s, &st)) return st;
  double* partial;
  int parts;
  st = norm_parts(grads, n_tensors, ord, ws, &partial, &parts, s);
  if (st != PRISM_OK) return st;
  if (parts == 0) {  // nothing but empty tensors
    finish_kernel<<<1, kGnThreads, 0, s>>>(partial, 0, ord == PRISM_NORM_INF, norm);
    return cuda_status(cudaGetLastError());
  }
  GnScale g = {partial, parts, ord == PRISM_NORM_INF, norm, 1, max_norm, eps};
  return n_tensors <= kFew ? run_scale<kFew>(grads, n_tensors, g, s) : run_scale<kMany>(grads, n_tensors, g, s);
}
