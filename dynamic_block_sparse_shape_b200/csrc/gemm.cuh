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
// Tiles. CG = 2: a pair of CTAs on neighbouring SMs computes 256 x BN: each
// holds 128 rows of A and half of B's rows, and the tensor cores of both read
// both halves of B, so a k-slice of 64 costs each SM 32 KB from L2 for 256 x 256
// x 64 / 2 multiply-adds (512 tensor cycles): 64 bytes per cycle and SM, where
// one CTA with a 128 x 256 tile would need 96. CG = 1: one CTA, 128 x BN, for
// products of few tiles.
//
// Roles of a CTA's six warps: 0 issues the copies into a ring of kStages
// slices; 1 owns the tensor memory and issues the products (of the pair: the
// leader's); 2..5 read the accumulator (a thread per row), apply the epilogue
// and store 32 x 64 tiles by TMA. Two accumulators: the epilogue of one tile
// runs beside the products of the next. Persistent CTAs walk the tiles in
// groups of kGroupM tile rows, whose operands then stay in L2.
#pragma once
#include "host.h"
#include "ptx.cuh"

namespace prism {

constexpr int kGemmM = 128;    // rows of A per CTA
constexpr int kGemmK = 64;     // a slice of K: one 128-byte swizzle row
constexpr int kGemmStages = 5;
constexpr int kGemmEpiWarps = 4;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;
constexpr int kGemmOutTile = 32 * 128;  // 32 rows x 64 bf16
constexpr int kGemmOutTiles = 3;        // per epilogue warp
constexpr int kGemmGroupM = 8;
constexpr int kGemmProducts = 3;

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
  int tiles_m, tiles_n, tile0;
  int slices0, slices;     // of segment 0, of both
};

struct GemmArgs {
  GemmProduct p[kGemmProducts];
  int products, tiles;
  int act, save;
  const __nv_bfloat16 *gate, *up;  // kEpiGateBwd: [m, n], contiguous
  int* status;
};

template <int CG, int BN>
struct GemmLayout {
  static constexpr int kA = kGemmM * 128;
  static constexpr int kB = BN / CG * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kOut = kGemmStages * kStage;
  static constexpr int kBars = kOut + kGemmEpiWarps * kGemmOutTiles * kGemmOutTile;
  static constexpr int kSmem = kBars + 256 + 1024;
  static constexpr int kCols = 2 * BN;  // tensor memory columns
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kCols <= 512, "tensor memory");
};

// ---------------------------------------------------------------- activations
// With e = exp(-z), sigmoid(z) = 1 / (1 + e) keeps its relative precision on
// either side of 0 (an infinite e gives 0).
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  if constexpr (ACT == PRISM_ACT_SILU) return g * sigmoid_f(g);
  // g Phi(g) through erfc, which has no cancellation where Phi is small
  if constexpr (ACT == PRISM_ACT_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
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
    const float p = 0.5f * erfcf(-0.70710678118654752f * g);
    a = g * p;
    slope = p + g * 0.39894228040143268f * __expf(-0.5f * g * g);
  } else if constexpr (ACT == PRISM_ACT_GELU_TANH) {
    const float s = sigmoid_f(1.5957691216057308f * (g + 0.044715f * g * g * g));
    a = g * s;
    slope = s + a * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * g * g);
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
// Arrives once on `bar` (of both CTAs of a pair) when this thread's products so far are complete.
template <int CG>
__device__ __forceinline__ void mma_commit_all(uint64_t* bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
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
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- the kernel
// Tile t of a launch: its product, tile row and tile column (groups of
// kGemmGroupM tile rows, tile column by tile column).
struct GemmTile {
  int product, tm, tn;
};
__device__ __forceinline__ GemmTile gemm_tile(const GemmArgs& P, int t) {
  GemmTile r;
  r.product = 0;
  while (r.product + 1 < P.products && t >= P.p[r.product + 1].tile0) ++r.product;
  const GemmProduct& Q = P.p[r.product];
  t -= Q.tile0;
  const int per = kGemmGroupM * Q.tiles_n, g = t / per;
  const int rows = min(kGemmGroupM, Q.tiles_m - g * kGemmGroupM);
  t -= g * per;
  r.tn = t / rows;
  r.tm = g * kGemmGroupM + (t - r.tn * rows);
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

// 32 bf16 values (packed) to half `half` of row `lane` of a 32 x 64 tile.
__device__ __forceinline__ void stage32(uint8_t* tile, int lane, int half, const uint32_t* w) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(tile + sw128_offset(lane, half * 4 + c)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// The epilogue of one 32-row, 64-column piece: columns `col` of the outputs,
// accumulator columns at `acc` (kEpiGate: u's at acc + BN / 2).
template <int BN, int EPI, int ACT>
__device__ __forceinline__ void gemm_piece(const GemmArgs& P, const GemmProduct& Q, uint32_t acc, uint8_t* tiles,
                                           int lane, int row, int col) {
  const bool row_in = row + lane < Q.m;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[32], w[16];
    if constexpr (EPI == kEpiStore) {
      tmem_ld32(acc + half * 32, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      stage32(tiles, lane, half, w);
    } else if constexpr (EPI == kEpiGate) {
      uint32_t u[32];
      tmem_ld32(acc + half * 32, r);
      tmem_ld32(acc + BN / 2 + half * 32, u);
      tmem_ld_wait();
      if (P.save) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        stage32(tiles + kGemmOutTile, lane, half, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        stage32(tiles + 2 * kGemmOutTile, lane, half, w);
      }
      // h from the fp32 projections, rounded once
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16x2(act_f<ACT>(__uint_as_float(r[2 * i])) * __uint_as_float(u[2 * i]),
                           act_f<ACT>(__uint_as_float(r[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
      stage32(tiles, lane, half, w);
    } else {
      // the saved projections of this row's 32 columns
      uint4 gv[4], uv[4];
      const size_t at = size_t(row + lane) * Q.n + col + half * 32;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = row_in && col + half * 32 + 8 * c < Q.n;
        gv[c] = in ? __ldg(reinterpret_cast<const uint4*>(P.gate + at) + c) : make_uint4(0, 0, 0, 0);
        uv[c] = in ? __ldg(reinterpret_cast<const uint4*>(P.up + at) + c) : make_uint4(0, 0, 0, 0);
      }
      tmem_ld32(acc + half * 32, r);
      tmem_ld_wait();
      uint32_t wg[16], wu[16];
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
      stage32(tiles, lane, half, wg);
      stage32(tiles + kGemmOutTile, lane, half, wu);
      if (P.save) stage32(tiles + 2 * kGemmOutTile, lane, half, w);
    }
  }
}

template <int CG, int BN, bool AMN, bool BMN, int EPI, int ACT>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs P) {
  using L = GemmLayout<CG, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBars);  // slice landed (leader's: of both CTAs)
  uint64_t* empty = full + kGemmStages;                         // slice's products complete
  uint64_t* acc_full = empty + kGemmStages;                     // [2] a tile's products complete
  uint64_t* acc_empty = acc_full + 2;                           // [2] accumulator read (leader's: by both CTAs)
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(mma_done + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
  int* status = P.status;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kGemmStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG * kGemmEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, L::kCols);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int t = cluster; t < P.tiles && ok; t += clusters) {
        const GemmTile T = gemm_tile(P, t);
        const GemmProduct& Q = P.p[T.product];
        const int row0 = (T.tm * CG + rank) * kGemmM;
        for (int kc = 0; kc < Q.slices; ++kc, ++it) {
          const int st = it % kGemmStages;
          if (it >= kGemmStages) ok = mbar_wait_abortable(&empty[st], ((it / kGemmStages) - 1) & 1, status, abort_flag);
          if (!ok) break;
          const int seg = kc >= Q.slices0;
          const int k0 = (kc - (seg ? Q.slices0 : 0)) * kGemmK;
          const uint32_t dst = smem_u32(sm + st * L::kStage);
          uint32_t bar = smem_u32(&full[st]);
          if constexpr (CG == 2) bar = map_shared(bar, 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], CG * L::kStage);
          gemm_load<CG, AMN>(dst, &Q.a[seg], bar, row0, k0, kGemmM);
          if constexpr (EPI == kEpiGate) {
            const int f0 = T.tn * (BN / 2);
            if constexpr (CG == 2) {
              gemm_load<CG, BMN>(dst + L::kA, &Q.b[rank], bar, f0, k0, BN / 2);
            } else {
              gemm_load<CG, BMN>(dst + L::kA, &Q.b[0], bar, f0, k0, BN / 2);
              gemm_load<CG, BMN>(dst + L::kA + BN / 2 * 128, &Q.b[1], bar, f0, k0, BN / 2);
            }
          } else {
            gemm_load<CG, BMN>(dst + L::kA, &Q.b[seg], bar, T.tn * BN + int(rank) * (BN / CG), k0, BN / CG);
          }
        }
      }
      // every copy has landed before a CTA may exit: the leader's barriers count both CTAs' copies
      if (rank == 0)
        for (int i = it > kGemmStages ? it - kGemmStages : 0; i < it; ++i)
          mbar_wait(&full[i % kGemmStages], (i / kGemmStages) & 1, status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(kGemmM * CG, BN, AMN, BMN);
      constexpr uint64_t kStepA = (AMN ? 2048 : 32) >> 4, kStepB = (BMN ? 2048 : 32) >> 4;  // 16 values of K
      bool ok = true;
      int it = 0, lt = 0;
      for (int t = cluster; t < P.tiles && ok; t += clusters, ++lt) {
        const int acc = lt & 1;
        if (lt >= 2) ok = mbar_wait_abortable(&acc_empty[acc], ((lt >> 1) - 1) & 1, status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tbase + acc * BN;
        const int slices = P.p[gemm_tile(P, t).product].slices;
        for (int kc = 0; kc < slices; ++kc, ++it) {
          const int st = it % kGemmStages;
          ok = mbar_wait_abortable(&full[st], (it / kGemmStages) & 1, status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(sm + st * L::kStage);
          // K-major: 8-row groups 1024 bytes apart; MN-major: 64-value boxes 8192 bytes apart, 8-k groups 1024
          const uint64_t da = sdesc_sw128(sa, AMN ? 8192 : 16, 1024), db = sdesc_sw128(sa + L::kA, BMN ? 8192 : 16, 1024);
#pragma unroll
          for (int k = 0; k < kGemmK / 16; ++k)
            mma_bf16<CG>(d, da + k * kStepA, db + k * kStepB, idesc, (kc > 0 || k > 0) ? 1u : 0u);
          mma_commit_all<CG>(&empty[st]);
        }
        if (ok) mma_commit_all<CG>(&acc_full[acc]);
      }
      // every product has completed before the tensor memory is released
      if constexpr (CG == 2) mma_commit_all<CG>(mma_done);
      else mma_commit(mma_done);
      mbar_wait(mma_done, 0, status);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // tensor memory lane quarter
    uint8_t* tiles = sm + L::kOut + (warp - 2) * kGemmOutTiles * kGemmOutTile;
    constexpr int kCols = EPI == kEpiGate ? BN / 2 : BN;  // output columns of a tile
    int lt = 0, ring = 0;
    for (int t = cluster; t < P.tiles; t += clusters, ++lt) {
      const GemmTile T = gemm_tile(P, t);
      const GemmProduct& Q = P.p[T.product];
      const int row = (T.tm * CG + int(rank)) * kGemmM + 32 * q, col0 = T.tn * kCols;
      const int acc = lt & 1;
      if (!mbar_wait_abortable(&acc_full[acc], (lt >> 1) & 1, status, abort_flag)) break;
      tc_fence_after();
      if (row < Q.m) {
#pragma unroll 1
        for (int c = 0; c < kCols && col0 + c < Q.n; c += 64) {
          // the tiles' last stores have been read: one tile a piece in a ring of three, or all three
          uint8_t* dst = tiles;
          if constexpr (EPI == kEpiStore) {
            dst = tiles + ring * kGemmOutTile;
            ring = ring == kGemmOutTiles - 1 ? 0 : ring + 1;
            if (lane == 0) bulk_wait_read<kGemmOutTiles - 1>();
          } else {
            if (lane == 0) bulk_wait_read<0>();
          }
          __syncwarp();
          gemm_piece<BN, EPI, ACT>(P, Q, tbase + acc * BN + (uint32_t(q * 32) << 16) + c, dst, lane, row, col0 + c);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const uint32_t src = smem_u32(dst);
            tma_store_2d(&Q.out[0], src, col0 + c, row);
            if (EPI == kEpiGateBwd || (EPI == kEpiGate && P.save))
              tma_store_2d(&Q.out[1], src + kGemmOutTile, col0 + c, row);
            if (EPI != kEpiStore && P.save) tma_store_2d(&Q.out[2], src + 2 * kGemmOutTile, col0 + c, row);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(map_shared(smem_u32(&acc_empty[acc]), 0));
        else mbar_arrive(&acc_empty[acc]);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  if constexpr (CG == 2) {
    // a pair that gave up may leave copies of the other CTA on their way: let them land
    if (*abort_flag) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000) {
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tbase, L::kCols);
  }
  if constexpr (CG == 2) cluster_sync_all();
}

}  // namespace prism
