// The bf16 matrix product behind the feed-forward block: D = A B^T with fp32
// accumulation in tensor memory and a fused epilogue, on tcgen05.
//
// Operands. A is [M, K], B is [N, K]; either lies in memory K-major (rows of K
// contiguous values) or MN-major (K rows of contiguous M or N values), which
// the tensor cores read equally fast, so no operand is ever transposed. A
// K-slice of 64 comes by TMA as 128-byte swizzled rows: [rows][64 k] K-major, or
// boxes of [64 k][64 mn] MN-major. What lies outside a tensor arrives as zeros.
// A product may run over two segments of K with operands of their own (dx =
// dg Wg + du Wu), and a launch may hold several products of the same kind (the
// three weight gradients).
//
// Tiles. What the tensor cores can be fed from L2 decides (measured: about 55
// bytes per cycle and SM at 1.5 GHz). A pair of CTAs on neighbouring SMs (CG = 2)
// computes 256 rows; each holds 128 rows of A and half of B's rows, and the
// tensor cores of both read both halves of B. SUB = 2: a tile is two
// accumulators of 256 columns that share A's slice, 256 x 512 in all: a slice
// of 64 k costs an SM 48 KB for 1024 tensor cycles, 48 bytes per cycle (64 with
// 256 x 256, 96 with one CTA's 128 x 256). Products of few tiles take the kernel
// of gemm_split.cuh, with single CTAs as well (CG = 1).
//
// Measured, 16384 x 4096 x 11264 with the power cap reached (the library's bf16
// product alone: 1439 TFLOP/s of 8192^3, 1322 to 1390 of these shapes): gate 1291
// TFLOP/s, down 1411, dx 1430, weight gradients 1418, the tensor pipe 88 to 95 %
// busy; gradient of the gate 1029 (70 %), whose SUB = 1 tiles and epilogue pieces (two
// [M, F] tensors read, three written) want 64 + 10 bytes per cycle and SM.
//
// Roles of a CTA's ten warps: 0 issues the copies into a ring of slices; 1
// owns the tensor memory and issues the products (of the pair: the leader's);
// 2..9 read the accumulators (a thread per row, two warps per row alternating
// over pieces of columns), apply the epilogue and store the pieces by TMA.
// SUB = 1: the two accumulators alternate, the epilogue of a tile runs beside
// the products of the next. SUB = 2: the next tile's first slices are
// multiplied into the first accumulator while the second is still being read.
// Persistent CTAs walk the tiles in groups of kGemmGroupM tile rows, whose
// operands then stay in L2; when the last round has work for less than half of
// the CTAs, its tiles are split into their two accumulators.
#pragma once
#include "host.h"
#include "ptx.cuh"

namespace prism {

constexpr int kGemmM = 128;    // rows of A per CTA
constexpr int kGemmK = 64;     // a slice of K: one 128-byte swizzle row
constexpr int kGemmEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;
constexpr int kGemmOutBytes = 4096;  // staging of an epilogue warp
// tile rows per group: 6 to 24 measured on blocks of 4096 to 32768 tokens, 12 best or within 1 %
constexpr int kGemmGroupM = 12;
constexpr int kGemmProducts = 3;
constexpr int kGemmMaxSmem = 232448;

// What happens to the accumulator.
enum GemmEpilogue : int {
  kEpiStore = 0,  // out 0 = D
  kEpiGate = 1,   // B's tile rows are half Wg, half Wu: out 0 = act(g) u, and with `save` out 1 = g, out 2 = u
  kEpiGateBwd = 2,  // D = dh: out 0 = dg, out 1 = du, and with `save` out 2 = h
};

struct GemmProduct {
  CUtensorMap a[2], b[2];  // by segment of K; kEpiGate: b[0] = Wg, b[1] = Wu
  CUtensorMap out[3];
  int m, n;                // rows and columns of the outputs
  int tiles_m, tiles_n;    // tile columns are of SUB accumulators
  int subs_n;              // accumulators over the columns
  int tile0;
  int slices0, slices;     // of segment 0, of both
};

struct GemmArgs {
  GemmProduct p[kGemmProducts];
  CUtensorMap in[2];  // kEpiGateBwd: the saved projections
  int products;
  int whole, units;   // tiles taken whole; these and the halves of the others
  int save;
  int follows;        // launched behind another product of the same call
  // reads nothing of the product it follows, which itself waited for all that both read before it let this one start:
  // runs beside it, and waits for it at the end alone, so that what comes next finds both complete
  int beside;
  // split kernel of single CTAs alone: kEpiGate (h) and kEpiGateBwd also write the bf16 remainders, m rows further on
  // (`fine`); kEpiStore adds row r + fold to row r and has `fold` rows
  int fine, fold;
  int* status;
};

// An epilogue piece is 32 rows x COLS bf16 values in swizzled rows: 64 columns
// (rows of 128 bytes: the copy engine's cost is by the row) where a warp stages
// one piece, 32 (rows of 64 bytes) where the gradient of the gate stages two
// and has two more coming in.
template <int COLS>
struct Piece {
  static constexpr int kBytes = 32 * COLS * 2, kSlots = kGemmOutBytes / kBytes, kChunks = COLS / 8;
  // byte offset of 16-byte chunk `chunk` of row `row`
  static __device__ __forceinline__ uint32_t offset(uint32_t row, uint32_t chunk) {
    return COLS == 64 ? sw128_offset(row, chunk) : row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
  }
};
constexpr int gemm_piece_cols(int epi) { return epi == kEpiGateBwd ? 32 : 64; }

constexpr int kPairN = 256;  // columns of an accumulator of the pair kernel

template <int SUB, int EPI>
struct GemmLayout {
  static constexpr int kA = kGemmM * 128;
  static constexpr int kB = kPairN / 2 * 128;
  static constexpr int kStage = kA + SUB * kB;
  static constexpr int kOutBytes = kGemmEpiWarps * kGemmOutBytes;
  static constexpr int kInBytes = EPI == kEpiGateBwd ? kGemmEpiWarps * 2 * Piece<32>::kBytes : 0;
  static constexpr int kFit = (kGemmMaxSmem - 1024 - 512 - kOutBytes - kInBytes) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kOut = kStages * kStage;
  static constexpr int kIn = kOut + kOutBytes;
  static constexpr int kBars = kIn + kInBytes;
  static constexpr int kSmem = kBars + 512 + 1024;
  static constexpr int kCols = 2 * kPairN;  // tensor memory columns
  static_assert(kSmem <= kGemmMaxSmem && kStages >= 3, "shared memory");
  static_assert(kCols <= 512, "tensor memory");
};

// What rounding v to the bf16 value `hi` left over (nothing of an infinity or NaN).
__device__ __forceinline__ float remainder_bf16(float v, float hi) {
  return fabsf(hi) < __int_as_float(0x7f800000) ? v - hi : 0.f;
}

// ---------------------------------------------------------------- activations
// With e = exp(-z), sigmoid(z) = 1 / (1 + e) keeps its relative precision on
// either side of 0 (an infinite e gives 0). The hardware's exponential and
// reciprocal (2 ulp and 1 ulp) do: the result is rounded to bf16.
__device__ __forceinline__ float sigmoid_f(float z) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// Phi(g) and exp(-g^2 / 2). With x = |g| / sqrt(2), erfc(x) = exp(-x^2) erfcx(x), and
// erfcx is smooth: a polynomial of degree 9 in t = 1 / (1 + x / 2), fitted to it
// over [0, 10.5] by reweighted least squares (relative error 4e-8, 3.3e-7 in fp32
// arithmetic). It keeps its relative precision where Phi is small, and the
// derivative shares its exponential; the library's erfc took three times as many
// instructions, which thin products (few values of K per output) waited for.
__device__ __forceinline__ void normal_f(float g, float& cdf, float& e) {
  const float x = fabsf(g) * 0.70710678118654752f;
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.5f, x, 1.f)));
  float p = -0.0591926179f;
  p = fmaf(p, t, 0.285179633f);
  p = fmaf(p, t, -0.488454836f);
  p = fmaf(p, t, 0.279506303f);
  p = fmaf(p, t, -0.0276195063f);
  p = fmaf(p, t, 0.203108422f);
  p = fmaf(p, t, 0.242996956f);
  p = fmaf(p, t, 0.282390025f);
  p = fmaf(p, t, 0.282085577f);
  const float q = 0.5f * e * (p * t);
  cdf = g < 0.f ? q : 1.f - q;
}

template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  if constexpr (ACT == PRISM_ACT_SILU) return g * sigmoid_f(g);
  if constexpr (ACT == PRISM_ACT_GELU) {
    float p, e;
    normal_f(g, p, e);
    return g * p;
  }
  // (1 + tanh z) / 2 = sigmoid(2 z)
  if constexpr (ACT == PRISM_ACT_GELU_TANH)
    return g * sigmoid_f(1.5957691216057308f * (g + 0.044715f * g * g * g));
  return g <= 0.f ? 0.f : g;  // NaN stays
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void act_slope_f(float g, float& a, float& slope) {
  if constexpr (ACT == PRISM_ACT_SILU) {
    const float s = sigmoid_f(g);
    a = g * s;
    slope = s + a * (1.f - s);
  } else if constexpr (ACT == PRISM_ACT_GELU) {
    float p, e;
    normal_f(g, p, e);
    a = g * p;
    slope = fmaf(g * 0.39894228040143268f, e, p);
  } else if constexpr (ACT == PRISM_ACT_GELU_TANH) {
    const float s = sigmoid_f(1.5957691216057308f * (g + 0.044715f * g * g * g));
    a = g * s;
    // s is 0 or 1 from |g| = 11 on, and 0 times an overflowed square would be NaN
    slope = s + a * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * fminf(g * g, 1e30f));
  } else {
    a = g <= 0.f ? 0.f : g;
    slope = g > 0.f ? 1.f : 0.f;
  }
}

// ---------------------------------------------------------------- PTX of pairs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barrier of every thread of the pair (release / acquire).
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address, in the cluster's shared window, of CTA `rank`'s object at this CTA's address.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// 2-D tiled load into this CTA's shared memory; the bytes are counted on the
// barrier at `bar` (CG = 2: the leader's). No multicast.
template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives once on `bar` (of both CTAs of a pair; `leader`: its even rank in the
// cluster) when this thread's products so far are complete.
template <int CG>
__device__ __forceinline__ void mma_commit_all(uint64_t* bar, uint32_t leader = 0) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3u << leader))
        : "memory");
  else
    mma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    tmem_dealloc(addr, cols);
}
// Programmatic dependent launch: waits for the kernels that this launch depends
// on (nothing when it was launched in plain stream order), and lets the next
// launch set itself up.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- the kernel
// Unit u of a launch's work: product, tile row, the first of its accumulators'
// columns and how many (groups of kGemmGroupM tile rows, tile column by tile
// column). Units from P.whole on are halves of tiles (an empty one where a tile
// has one accumulator only).
struct GemmUnit {
  int product, tm, sub, subs;
};
template <int SUB>
__device__ __forceinline__ GemmUnit gemm_unit(const GemmArgs& P, int u) {
  const bool half = SUB == 2 && u >= P.whole;
  int t = half ? P.whole + ((u - P.whole) >> 1) : u;
  GemmUnit r;
  r.product = 0;
  while (r.product + 1 < P.products && t >= P.p[r.product + 1].tile0) ++r.product;
  const GemmProduct& Q = P.p[r.product];
  t -= Q.tile0;
  const int per = kGemmGroupM * Q.tiles_n, g = t / per;
  const int rows = min(kGemmGroupM, Q.tiles_m - g * kGemmGroupM);
  t -= g * per;
  const int tn = t / rows;
  r.tm = g * kGemmGroupM + (t - tn * rows);
  r.sub = tn * SUB + (half ? (u - P.whole) & 1 : 0);
  r.subs = max(0, min(half ? 1 : SUB, Q.subs_n - r.sub));
  return r;
}

// `rows` rows (a multiple of 64 when MN-major) of a K-slice into shared memory.
template <int CG, bool MN>
__device__ __forceinline__ void gemm_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int mn0, int k0, int rows) {
  if constexpr (MN) {
    for (int r = 0; r < rows; r += 64) tma_load_2d<CG>(dst + r * 128, map, bar, mn0 + r, k0);
  } else {
    tma_load_2d<CG>(dst, map, bar, k0, mn0);
  }
}

// An epilogue warp's staging: pieces leave by TMA stores, each waited for
// (until read) before its place is written again.
template <int COLS>
struct PieceRing {
  uint8_t* base;
  int at;
  // f(i, w): 16 packed words of this lane's row, columns 32 i to 32 i + 31
  template <typename F>
  __device__ __forceinline__ void store(const CUtensorMap* map, int lane, int row, int col, const F& f) {
    uint8_t* p = base + at * Piece<COLS>::kBytes;
    at = at + 1 == Piece<COLS>::kSlots ? 0 : at + 1;
    if (lane == 0) bulk_wait_read<Piece<COLS>::kSlots - 1>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < COLS / 32; ++i) {
      uint32_t w[16];
      f(i, w);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(p + Piece<COLS>::offset(lane, 4 * i + c)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, smem_u32(p), col, row);
      bulk_commit_group();
    }
  }
};

__device__ __forceinline__ void pack32(const uint32_t* r, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// kEpiStore, kEpiGate: the outputs of one 32-row, 64-column piece from its
// accumulator values r (kEpiGate: of g, and u of u).
template <int EPI, int ACT>
__device__ __forceinline__ void gemm_piece(const GemmArgs& P, const GemmProduct& Q, const uint32_t* r, const uint32_t* u,
                                           PieceRing<64>& ring, int lane, int row, int col) {
  if constexpr (EPI == kEpiStore) {
    ring.store(&Q.out[0], lane, row, col, [&](int i, uint32_t* w) { pack32(r + 32 * i, w); });
  } else {
    // h from the fp32 projections, rounded once
    ring.store(&Q.out[0], lane, row, col, [&](int i, uint32_t* w) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int x = 32 * i + 2 * j;
        w[j] = pack_bf16x2(act_f<ACT>(__uint_as_float(r[x])) * __uint_as_float(u[x]),
                           act_f<ACT>(__uint_as_float(r[x + 1])) * __uint_as_float(u[x + 1]));
      }
    });
    if (P.save) {
      ring.store(&Q.out[1], lane, row, col, [&](int i, uint32_t* w) { pack32(r + 32 * i, w); });
      ring.store(&Q.out[2], lane, row, col, [&](int i, uint32_t* w) { pack32(u + 32 * i, w); });
    }
  }
}

__device__ __forceinline__ void copy16(const uint32_t* from, uint32_t* to) {
#pragma unroll
  for (int i = 0; i < 16; ++i) to[i] = from[i];
}

// kEpiGateBwd: the outputs of one 32-row, 32-column piece from dh in tensor
// memory at `acc` and the saved projections' piece at `in` (gate, then up);
// `taken` once that is read, which lets the next piece be copied over it. That
// comes behind the first output's store, not behind the loads: a warp goes on
// while its loads of shared memory still queue (behind the load of tensor memory),
// and a copy need not wait for them. The first output holds every value of the
// piece, so that its stores are issued shows that all loads are back; the fence in
// there orders them against the copy.
template <int ACT, typename F>
__device__ __forceinline__ void gemm_piece_bwd(const GemmArgs& P, const GemmProduct& Q, uint32_t acc, PieceRing<32>& ring,
                                               const uint8_t* in, int lane, int row, int col, const F& taken) {
  uint32_t r[32], w[16], wg[16], wu[16];
  uint4 gv[4], uv[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    gv[c] = *reinterpret_cast<const uint4*>(in + Piece<32>::offset(lane, c));
    uv[c] = *reinterpret_cast<const uint4*>(in + Piece<32>::kBytes + Piece<32>::offset(lane, c));
  }
  tmem_ld32(acc, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t g2 = reinterpret_cast<const uint32_t*>(gv)[i], u2 = reinterpret_cast<const uint32_t*>(uv)[i];
    float dg[2], du[2], h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float g = __uint_as_float(e ? g2 & 0xFFFF0000u : g2 << 16);
      const float u = __uint_as_float(e ? u2 & 0xFFFF0000u : u2 << 16);
      const float dh = __uint_as_float(r[2 * i + e]);
      float a, s;
      act_slope_f<ACT>(g, a, s);
      dg[e] = dh * u * s;
      du[e] = dh * a;
      h[e] = a * u;
    }
    wg[i] = pack_bf16x2(dg[0], dg[1]);
    wu[i] = pack_bf16x2(du[0], du[1]);
    w[i] = pack_bf16x2(h[0], h[1]);
  }
  ring.store(&Q.out[0], lane, row, col, [&](int, uint32_t* x) { copy16(wg, x); });
  taken();
  ring.store(&Q.out[1], lane, row, col, [&](int, uint32_t* x) { copy16(wu, x); });
  if (P.save) ring.store(&Q.out[2], lane, row, col, [&](int, uint32_t* x) { copy16(w, x); });
}

template <int SUB, bool AMN, bool BMN, int EPI, int ACT>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs P) {
  using L = GemmLayout<SUB, EPI>;
  constexpr int CG = 2, BN = kPairN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBars);  // slice landed (leader's: of both CTAs)
  uint64_t* empty = full + L::kStages;                          // slice's products complete
  uint64_t* acc_full = empty + L::kStages;                      // [2] an accumulator's products complete
  uint64_t* acc_empty = acc_full + 2;                           // [2] accumulator read (leader's: by both CTAs)
  uint64_t* mma_done = acc_empty + 2;
  uint64_t* in_full = mma_done + 1;                             // [epilogue warps] saved projections landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + kGemmEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
  int* status = P.status;
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&P.p[0].a[0]);
    tma_prefetch_desc(&P.p[0].b[0]);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG * kGemmEpiWarps);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < kGemmEpiWarps; ++i) mbar_init(&in_full[i], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, L::kCols);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  if (!P.beside) grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int u = cluster; u < P.units && ok; u += clusters) {
        const GemmUnit U = gemm_unit<SUB>(P, u);
        if (U.subs == 0) continue;
        const GemmProduct& Q = P.p[U.product];
        const int row0 = (U.tm * CG + rank) * kGemmM;
        for (int kc = 0; kc < Q.slices; ++kc, ++it) {
          const int st = it % L::kStages;
          if (it >= L::kStages) ok = mbar_wait_abortable(&empty[st], ((it / L::kStages) - 1) & 1, status, abort_flag);
          if (!ok) break;
          const int seg = kc >= Q.slices0;
          const int k0 = (kc - (seg ? Q.slices0 : 0)) * kGemmK;
          uint32_t dst = smem_u32(sm + st * L::kStage);
          const uint32_t bar = map_shared(smem_u32(&full[st]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], CG * (L::kA + U.subs * L::kB));
          gemm_load<CG, AMN>(dst, &Q.a[seg], bar, row0, k0, kGemmM);
          dst += L::kA;
          for (int i = 0; i < U.subs; ++i, dst += L::kB) {
            if constexpr (EPI == kEpiGate) {
              const int f0 = (U.sub + i) * (BN / 2);
              gemm_load<CG, BMN>(dst, &Q.b[rank], bar, f0, k0, BN / 2);
            } else {
              gemm_load<CG, BMN>(dst, &Q.b[seg], bar, (U.sub + i) * BN + int(rank) * (BN / CG), k0, BN / CG);
            }
          }
        }
      }
      // every copy has landed before a CTA may exit: the leader's barriers count both CTAs' copies
      if (rank == 0)
        for (int i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
          mbar_wait(&full[i % L::kStages], (i / L::kStages) & 1, status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(kGemmM * CG, BN, AMN, BMN);
      constexpr uint64_t kStepA = (AMN ? 2048 : 32) >> 4, kStepB = (BMN ? 2048 : 32) >> 4;  // 16 values of K
      // slice in ring place st, times B's rows of accumulator `sub`; K-major: 8-row groups 1024 bytes apart;
      // MN-major: 64-value boxes 8192 bytes apart, 8-k groups 1024
      auto multiply = [&](int st, int sub, uint32_t d, bool first) {
        const uint32_t sa = smem_u32(sm + st * L::kStage);
        const uint64_t da = sdesc_sw128(sa, AMN ? 8192 : 16, 1024);
        const uint64_t db = sdesc_sw128(sa + L::kA + sub * L::kB, BMN ? 8192 : 16, 1024);
#pragma unroll
        for (int k = 0; k < kGemmK / 16; ++k)
          mma_bf16<CG>(d, da + k * kStepA, db + k * kStepB, idesc, (!first || k > 0) ? 1u : 0u);
      };
      bool ok = true;
      int it = 0, j = 0;  // slices, accumulators so far
      for (int u = cluster; u < P.units && ok; u += clusters) {
        const GemmUnit U = gemm_unit<SUB>(P, u);
        if (U.subs == 0) continue;
        const int slices = P.p[U.product].slices;
        const int acc = j & 1;
        const uint32_t d0 = tbase + acc * BN, d1 = tbase + (acc ^ 1) * BN;
        if (j >= 2) ok = mbar_wait_abortable(&acc_empty[acc], ((j >> 1) - 1) & 1, status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        int kc = 0;
        if (SUB == 2 && U.subs == 2) {
          // the first slices into the first accumulator, while the second may still be read
          const int pre = min(slices, L::kStages);
          for (; kc < pre; ++kc) {
            ok = mbar_wait_abortable(&full[(it + kc) % L::kStages], ((it + kc) / L::kStages) & 1, status, abort_flag);
            if (!ok) break;
            tc_fence_after();
            multiply((it + kc) % L::kStages, 0, d0, kc == 0);
            if (kc == slices - 1) mma_commit_all<CG>(&acc_full[acc]);
          }
          if (!ok) break;
          if (j + 1 >= 2) ok = mbar_wait_abortable(&acc_empty[acc ^ 1], (((j + 1) >> 1) - 1) & 1, status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          for (kc = 0; kc < pre; ++kc, ++it) {
            multiply(it % L::kStages, 1, d1, kc == 0);
            mma_commit_all<CG>(&empty[it % L::kStages]);
          }
        }
        for (; kc < slices; ++kc, ++it) {
          const int st = it % L::kStages;
          ok = mbar_wait_abortable(&full[st], (it / L::kStages) & 1, status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          multiply(st, 0, d0, kc == 0);
          if (kc == slices - 1) mma_commit_all<CG>(&acc_full[acc]);
          if (SUB == 2 && U.subs == 2) multiply(st, 1, d1, false);
          mma_commit_all<CG>(&empty[st]);
        }
        if (ok && U.subs == 2) mma_commit_all<CG>(&acc_full[acc ^ 1]);
        j += U.subs;
      }
      // every product has completed before the tensor memory is released
      mma_commit_all<CG>(mma_done);
      mbar_wait(mma_done, 0, status);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;           // tensor memory lane quarter
    const int e = warp - 2;
    constexpr int kPiece = gemm_piece_cols(EPI);
    const int c0 = (e >> 2) * kPiece;  // of the two warps of a quarter, one takes the even pieces, one the odd
    PieceRing<kPiece> ring = {sm + L::kOut + e * kGemmOutBytes, 0};
    uint8_t* in = sm + L::kIn + e * 2 * Piece<32>::kBytes;  // gate, up
    uint64_t* in_bar = in_full + e;
    constexpr int kCols = EPI == kEpiGate ? BN / 2 : BN;  // output columns of an accumulator
    constexpr int kMine = kCols / (2 * kPiece);           // pieces of this warp
    int j = 0, pieces = 0;
    bool ok = true;
    for (int u = cluster; u < P.units && ok; u += clusters) {
      const GemmUnit U = gemm_unit<SUB>(P, u);
      const GemmProduct& Q = P.p[U.product];
      const int row = (U.tm * CG + int(rank)) * kGemmM + 32 * q;
      for (int i = 0; i < U.subs; ++i, ++j) {
        const int col = (U.sub + i) * kCols, acc = j & 1;
        const int end = row < Q.m ? min(kCols, Q.n - col) : 0;
        const uint32_t t_acc = tbase + acc * BN + (uint32_t(q * 32) << 16) + c0;
        auto wait_acc = [&]() {
          ok = __all_sync(0xffffffffu, mbar_wait_abortable(&acc_full[acc], (j >> 1) & 1, status, abort_flag));
          tc_fence_after();
          return ok;
        };
        auto release_acc = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_shared(smem_u32(&acc_empty[acc]), 0));
        };
        if constexpr (EPI == kEpiGateBwd) {
          auto fetch = [&](int c) {  // the saved projections of the piece at column c
            if (c < end && lane == 0) {
              mbar_arrive_expect_tx(in_bar, 2 * Piece<32>::kBytes);
              tma_load_2d<1>(smem_u32(in), &P.in[0], smem_u32(in_bar), col + c, row);
              tma_load_2d<1>(smem_u32(in) + Piece<32>::kBytes, &P.in[1], smem_u32(in_bar), col + c, row);
            }
          };
          fetch(c0);
          if (!wait_acc()) break;
#pragma unroll 1
          for (int c = c0; c < end; c += 2 * kPiece, ++pieces) {
            ok = __all_sync(0xffffffffu, mbar_wait_abortable(in_bar, pieces & 1, status, abort_flag));
            if (!ok) break;
            gemm_piece_bwd<ACT>(P, Q, t_acc + (c - c0), ring, in, lane, row, col + c,
                                [&]() { fetch(c + 2 * kPiece); });
          }
          if (!ok) break;
          release_acc();
        } else {
          // all of this warp's values into registers, so that the accumulator is free at once
          if (!wait_acc()) break;
          uint32_t r[kMine][kPiece], v[EPI == kEpiGate ? kMine : 1][kPiece];
#pragma unroll
          for (int p = 0; p < kMine; ++p)
#pragma unroll
            for (int x = 0; x < kPiece; x += 32) {
              tmem_ld32(t_acc + p * 2 * kPiece + x, r[p] + x);
              if constexpr (EPI == kEpiGate) tmem_ld32(t_acc + BN / 2 + p * 2 * kPiece + x, v[p] + x);
            }
          tmem_ld_wait();
          release_acc();
#pragma unroll
          for (int p = 0; p < kMine; ++p) {
            const int c = c0 + p * 2 * kPiece;
            if (c < end) gemm_piece<EPI, ACT>(P, Q, r[p], v[EPI == kEpiGate ? p : 0], ring, lane, row, col + c);
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  // a CTA that gave up may leave copies of its own or of its pair on their way: let them land
  if (*abort_flag) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000) {
    }
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tbase, L::kCols);
  }
  cluster_sync_all();
  if (P.beside) grid_dependency_wait();
}

}  // namespace prism
