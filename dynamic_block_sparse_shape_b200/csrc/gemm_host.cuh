// Host side of gemm.cuh: tensor maps, the choice of tiles, the launch.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gemm_split.cuh"

namespace prism {

// Rows of a matrix in memory: `mn` rows (or columns, MN-major) against `k`.
struct GemmOperand {
  const void* base = nullptr;
  int64_t ld = 0;  // elements between rows in memory
};
struct GemmOutput {
  void* base = nullptr;
  int64_t ld = 0;
};
struct GemmProblem {
  GemmOperand a[2], b[2];
  GemmOutput out[3];
  const void* in[2] = {nullptr, nullptr};  // kEpiGateBwd: the saved projections, contiguous
  int64_t m = 0, n = 0;
  int64_t k[2] = {0, 0};
};

inline prism_status gemm_operand_map(CUtensorMap* map, const GemmOperand& o, bool mn_major, int64_t mn, int64_t k,
                                     int box_rows) {
  const uint64_t dims[2] = {uint64_t(mn_major ? mn : k), uint64_t(mn_major ? k : mn)};
  const uint64_t strides[1] = {uint64_t(o.ld) * 2};
  const uint32_t box[2] = {64, uint32_t(mn_major ? 64 : box_rows)};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A piece of 32 rows of an [m, n] matrix, as the epilogue reads and writes it.
inline prism_status gemm_piece_map(CUtensorMap* map, const void* base, int64_t m, int64_t n, int64_t ld, int cols) {
  const uint64_t dims[2] = {uint64_t(n), uint64_t(m)};
  const uint64_t strides[1] = {uint64_t(ld) * 2};
  const uint32_t box[2] = {uint32_t(cols), 32};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
                      cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// The launch's attributes: the cluster, and for a product that follows another
// of the same call (P.follows) a programmatic dependence on it, so that its
// launch and setup run beside the other's end.
inline void gemm_follow(const GemmArgs& P, cudaLaunchAttribute* at, int n, cudaLaunchConfig_t* cfg) {
  if (P.follows) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg->attrs = at;
  cfg->numAttrs = n;
}

template <int SUB, bool AMN, bool BMN, int EPI, int ACT>
prism_status gemm_launch(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s) {
  using L = GemmLayout<SUB, EPI>;
  constexpr int CG = 2, BN = kPairN;
  constexpr int kCols = EPI == kEpiGate ? BN / 2 : BN;
  constexpr int kRowsB = EPI == kEpiGate ? BN / 2 : BN / CG;
  P.products = products;
  int tiles = 0;
  for (int i = 0; i < products; ++i) {
    GemmProduct& Q = P.p[i];
    const GemmProblem& R = pr[i];
    Q.m = int(R.m);
    Q.n = int(R.n);
    Q.tiles_m = int((R.m + kGemmM * CG - 1) / (kGemmM * CG));
    Q.subs_n = int((R.n + kCols - 1) / kCols);
    Q.tiles_n = (Q.subs_n + SUB - 1) / SUB;
    Q.tile0 = tiles;
    if (int64_t(Q.tiles_m) * Q.tiles_n + tiles > (int64_t(1) << 29)) return PRISM_ERR_UNSUPPORTED;
    tiles += Q.tiles_m * Q.tiles_n;
    Q.slices0 = int((R.k[0] + kGemmK - 1) / kGemmK);
    Q.slices = Q.slices0 + int((R.k[1] + kGemmK - 1) / kGemmK);
    prism_status st = PRISM_OK;
    for (int g = 0; g < 2 && st == PRISM_OK; ++g) {
      if (R.a[g].base) st = gemm_operand_map(&Q.a[g], R.a[g], AMN, R.m, R.k[g], kGemmM);
      const int64_t kb = EPI == kEpiGate ? R.k[0] : R.k[g];
      if (R.b[g].base && st == PRISM_OK) st = gemm_operand_map(&Q.b[g], R.b[g], BMN, R.n, kb, kRowsB);
    }
    for (int g = 0; g < 3 && st == PRISM_OK; ++g)
      if (R.out[g].base) st = gemm_piece_map(&Q.out[g], R.out[g].base, R.m, R.n, R.out[g].ld, gemm_piece_cols(EPI));
    if (st != PRISM_OK) return st;
  }
  if constexpr (EPI == kEpiGateBwd) {
    prism_status st = PRISM_OK;
    for (int g = 0; g < 2 && st == PRISM_OK; ++g) st = gemm_piece_map(&P.in[g], pr[0].in[g], pr[0].m, pr[0].n, pr[0].n,
                                                                      gemm_piece_cols(EPI));
    if (st != PRISM_OK) return st;
  }
  int clusters = device_sm_count() / CG;
  P.whole = tiles;
  if (SUB == 2 && tiles % clusters * 2 <= clusters) P.whole = tiles / clusters * clusters;
  P.units = P.whole + 2 * (tiles - P.whole);
  if (clusters > P.units) clusters = P.units;
  auto kernel = gemm_kernel<SUB, AMN, BMN, EPI, ACT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) != cudaSuccess)
    return PRISM_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(clusters * CG);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  gemm_follow(P, at, 1, &cfg);
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P));
}

// CTAs that run at once in clusters of `ranks`, one or two per SM: a cluster
// stays within a group of SMs, and what is left over of the groups stays idle
// (as the occupancy query says for a B200: 148, 148, 132, 120 CTAs in clusters of
// 1, 2, 4, 8 at one per SM, 296, 296, 284, 264 at two).
inline int64_t split_slots(int ranks, int per_sm) {
  const int idle = ranks >= 8 ? (per_sm == 1 ? 28 : 32) : ranks >= 4 ? (per_sm == 1 ? 16 : 12) : 0;
  return int64_t(device_sm_count()) * per_sm - idle;
}

constexpr int kSplitHalf = 113 * 1024;  // shared memory of each of two CTAs on an SM

inline int split_slot_rows(int a_rows, int fold, int parts) {
  return fold ? 2 * ((fold + parts - 1) / parts) : (a_rows + parts - 1) / parts;
}

template <int CG, int BN, bool AMN, bool BMN, int EPI, int ACT>
prism_status gemm_split_launch(const GemmArgs& P, const GemmProblem* pr, int products, int parts, cudaStream_t s) {
  constexpr int kCols = EPI == kEpiGate ? BN / 2 : BN;
  SplitLaunch A;
  std::memset(&A, 0, sizeof(A));
  A.products = products;
  A.save = P.save;
  A.beside = P.beside;
  A.fine = P.fine;
  A.fold = P.fold;
  A.status = P.status;
  const int a_rows = AMN || CG == 2 || pr[0].m >= kGemmM ? kGemmM : int(pr[0].m + 7) / 8 * 8;
  A.a_bytes = a_rows * 128;
  int64_t tiles = 0, slices = 0;
  for (int i = 0; i < products; ++i) {
    SplitArgs& Q = A.p[i];
    const GemmProblem& R = pr[i];
    Q.m = int(R.m);
    Q.n = int(R.n);
    Q.tiles_m = int((R.m + CG * kGemmM - 1) / (CG * kGemmM));
    Q.tiles_n = int((R.n + kCols - 1) / kCols);
    Q.tile0 = int(tiles);
    tiles += int64_t(Q.tiles_m) * Q.tiles_n;
    Q.slices0 = int((R.k[0] + kGemmK - 1) / kGemmK);
    Q.slices = Q.slices0 + int((R.k[1] + kGemmK - 1) / kGemmK);
    if (Q.slices > slices) slices = Q.slices;
    prism_status st = PRISM_OK;
    for (int g = 0; g < 2 && st == PRISM_OK; ++g) {
      if (R.a[g].base) st = gemm_operand_map(&Q.a[g], R.a[g], AMN, R.m, R.k[g], a_rows);
      const int64_t kb = EPI == kEpiGate ? R.k[0] : R.k[g];
      if (R.b[g].base && st == PRISM_OK) st = gemm_operand_map(&Q.b[g], R.b[g], BMN, R.n, kb, EPI == kEpiGate ? BN / 2 : BN / CG);
      Q.in[g] = static_cast<const __nv_bfloat16*>(R.in[g]);
    }
    if (st != PRISM_OK) return st;
    for (int g = 0; g < 3; ++g) {
      Q.out[g] = static_cast<__nv_bfloat16*>(R.out[g].base);
      Q.out_ld[g] = R.out[g].ld;
    }
  }
  const int ranks = CG * parts;
  if (tiles * ranks >= (int64_t(1) << 31)) return PRISM_ERR_UNSUPPORTED;
  // a ring of all of an SM's shared memory, or two of half of it
  A.slot_rows = split_slot_rows(a_rows, P.fold, parts);
  const auto need = [&](int stages) { return split_smem(CG, BN, A.a_bytes, stages, parts, A.slot_rows); };
  const int room = CG == 2 || tiles * ranks <= split_slots(ranks, 1) || need(1) > kSplitHalf ? kGemmMaxSmem : kSplitHalf;
  A.stages = int(std::min<int64_t>(kSplitStages, (slices + parts - 1) / parts));
  while (A.stages > 1 && need(A.stages) > room) --A.stages;
  const int smem = need(A.stages);
  if (smem > room) return PRISM_ERR_UNSUPPORTED;  // see gemm_choice
  auto kernel = gemm_split_kernel<CG, BN, AMN, BMN, EPI, ACT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmMaxSmem) != cudaSuccess)
    return PRISM_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned(tiles * ranks));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  gemm_follow(P, at, 1, &cfg);
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, A));
}

// Time of a product in ns by what it is made of (fitted to the measured times of
// ten choices each for the products of 13 sizes of 33 to 3000 rows; the choices it
// takes are 0.9 % behind the best ones in the mean, 14 % at worst): an SM fetches
// kRate bytes per ns from L2, rows that do not start on 128-byte borders count
// kRagged times; a slice takes at least its tensor cycles and a CTA kSliceNs, and
// a ring's slices come back after kLatencyNs; a tile's fill and epilogue, of a
// single CTA, a pair, and the persistent pairs; and the joining of parts.
constexpr double kRate = 90.0, kRagged = 1.3, kLatencyNs = 1200.0, kSliceNs = 350.0, kCycleNs = 1.0 / 1.7,
                 kTileNs = 4500.0, kPairTileNs = 6000.0, kPersistentNs = 5000.0, kJoinNs = 300.0, kJoinRate = 40.0;

struct GemmChoice {
  int cg, bn, parts;  // bn = 0: the pair kernel of gemm.cuh
};

// The kernel and tiles for products of m x n rows each (n: columns of the
// accumulator): the choice of least time by the figures above; what they are
// off by shows only where two choices are close. `sub`: accumulators of a tile
// of the pair kernel; `single`: single CTAs only (what the pairs' epilogue lacks).
inline GemmChoice gemm_choice(const int64_t* m, const int64_t* n, int products, int64_t slices, bool a_mn, int sub,
                              bool ragged, bool single) {
  const int sms = device_sm_count();
  auto tiles = [&](int64_t rows, int64_t cols) {
    double t = 0;
    for (int i = 0; i < products; ++i) t += double((m[i] + rows - 1) / rows) * double((n[i] + cols - 1) / cols);
    return t;
  };
  const double rate = ragged ? kRate / kRagged : kRate, k = double(slices);
  // pairs: rounds of tiles, the last one of single accumulators when it is less than half full
  const double pairs = sms / 2, accs = tiles(256, 256);
  const double whole = std::floor(accs / sub / pairs), rest = accs / sub - whole * pairs;
  const double one = std::fmax(32768.0 / rate, 512 * kCycleNs);
  const double both = sub == 1 ? one : std::fmax(49152.0 / rate, 1024 * kCycleNs);
  double best = k * (whole * both + (rest > 0 ? (rest * 2 <= pairs ? one : both) : 0.0)) + kPersistentNs;
  GemmChoice c = {2, 0, 1};
  if (single) best = HUGE_VAL;
  // with the most parts that shared memory has room for: of four parts of a pair's tile not even the sums fit
  const GemmChoice tries[] = {{1, 64, 8}, {1, 128, 4}, {2, 256, 2}};
  for (const GemmChoice& t : tries) {
    if (single && t.cg == 2) continue;
    const int rows_a = a_mn || t.cg == 2 || m[0] >= kGemmM ? kGemmM : int(m[0] + 7) / 8 * 8;
    const double bytes = (rows_a + t.bn / t.cg) * 128.0;
    for (int parts = 1; parts <= t.parts && parts <= slices; parts *= 2) {
      const int least = split_smem(t.cg, t.bn, rows_a * 128, 1, parts, split_slot_rows(rows_a, 0, parts) + 1);
      if (least > kGemmMaxSmem) continue;
      const int64_t ctas = int64_t(tiles(kGemmM * t.cg, t.bn)) * t.cg * parts, one_each = split_slots(t.cg * parts, 1);
      // rounds of CTAs, and how many an SM works through in all
      int64_t rounds = (ctas + one_each - 1) / one_each, load = rounds;
      if (t.cg == 1 && rounds > 1 && least <= kSplitHalf) {
        const int64_t two_each = split_slots(parts, 2);
        rounds = (ctas + two_each - 1) / two_each;
        load = 2 * rounds - (ctas - (rounds - 1) * two_each <= one_each);
      }
      const double mine = std::ceil(k / parts);
      const double flight = std::fmin(std::fmin(mine, double(kSplitStages)) * (t.cg == 1 && load > 1 ? 2.0 : 1.0),
                                      kGemmMaxSmem / bytes);
      const double slice = std::fmax(std::fmax(bytes / rate, load > rounds ? kSliceNs / 2 : kSliceNs), kLatencyNs / std::fmax(flight, 1.0));
      const double join = parts > 1 ? double(rounds) * kJoinNs + double(load) * rows_a * t.bn * 4.0 / kJoinRate : 0.0;
      const double ns = double(load) * mine * slice + double(rounds) * (t.cg == 2 ? kPairTileNs : kTileNs) + join;
      if (ns < best) {
        best = ns;
        c = {t.cg, t.bn, parts};
      }
    }
  }
  return c;
}

// `form`: only says which kernel and tiles it would take.
template <bool AMN, bool BMN, int EPI, int ACT>
prism_status gemm(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s, GemmChoice* form) {
  // the gradient of the gate has the longest epilogue: it alternates its accumulators to hide it
  constexpr int kSub = EPI == kEpiGateBwd ? 1 : 2;
  int64_t m[kGemmProducts], n[kGemmProducts], slices = 0;
  bool ragged = false;
  for (int i = 0; i < products; ++i) {
    m[i] = pr[i].m;
    n[i] = pr[i].n * (EPI == kEpiGate ? 2 : 1);
    slices = std::max(slices, (pr[i].k[0] + kGemmK - 1) / kGemmK + (pr[i].k[1] + kGemmK - 1) / kGemmK);
    ragged = ragged || pr[i].a[0].ld % 64 || pr[i].b[0].ld % 64;
  }
  const GemmChoice c = gemm_choice(m, n, products, slices, AMN, kSub, ragged, P.fine || P.fold);
  if (form) {
    *form = c;
    return PRISM_OK;
  }
  if (c.bn == 0) return gemm_launch<kSub, AMN, BMN, EPI, ACT>(P, pr, products, s);
  if (c.cg == 1 && c.bn == 64) return gemm_split_launch<1, 64, AMN, BMN, EPI, ACT>(P, pr, products, c.parts, s);
  if (c.cg == 1) return gemm_split_launch<1, 128, AMN, BMN, EPI, ACT>(P, pr, products, c.parts, s);
  return gemm_split_launch<2, 256, AMN, BMN, EPI, ACT>(P, pr, products, c.parts, s);
}

}  // namespace prism
