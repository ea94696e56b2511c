// Host side of gemm.cuh: tensor maps, the choice of tiles, the launch.
#pragma once
#include <cstring>

#include "gemm.cuh"

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

// A 32 x 32 piece of an [m, n] matrix, as the epilogue reads and writes it.
inline prism_status gemm_piece_map(CUtensorMap* map, const void* base, int64_t m, int64_t n, int64_t ld) {
  const uint64_t dims[2] = {uint64_t(n), uint64_t(m)};
  const uint64_t strides[1] = {uint64_t(ld) * 2};
  const uint32_t box[2] = {kGemmPiece, 32};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int CG, int BN, int SUB, bool AMN, bool BMN, int EPI, int ACT>
prism_status gemm_launch(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s) {
  using L = GemmLayout<CG, BN, SUB, EPI>;
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
      if (R.out[g].base) st = gemm_piece_map(&Q.out[g], R.out[g].base, R.m, R.n, R.out[g].ld);
    if (st != PRISM_OK) return st;
  }
  int clusters = device_sm_count() / CG;
  P.whole = tiles;
  if (SUB == 2 && tiles % clusters * 2 <= clusters) P.whole = tiles / clusters * clusters;
  P.units = P.whole + 2 * (tiles - P.whole);
  if (clusters > P.units) clusters = P.units;
  auto kernel = gemm_kernel<CG, BN, SUB, AMN, BMN, EPI, ACT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) != cudaSuccess)
    return PRISM_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(clusters * CG);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CG > 1 ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P));
}

// Pairs of CTAs when there is an accumulator of 256 x 256 for each of the SMs'
// pairs; otherwise smaller tiles of single CTAs, as many as possible.
template <bool AMN, bool BMN, int EPI, int ACT>
prism_status gemm(GemmArgs& P, const GemmProblem* pr, int products, cudaStream_t s) {
  const int sms = device_sm_count();
  auto tiles = [&](int rows, int cols) {
    int64_t t = 0;
    for (int i = 0; i < products; ++i) t += ((pr[i].m + rows - 1) / rows) * ((pr[i].n + cols - 1) / cols);
    return t;
  };
  constexpr int kHalf = EPI == kEpiGate ? 2 : 1;
  // the gradient of the gate has the longest epilogue: it needs the second accumulator to hide it
  constexpr int kSub = EPI == kEpiGateBwd ? 1 : 2;
  if (tiles(256, 256 / kHalf) * 2 >= sms) return gemm_launch<2, 256, kSub, AMN, BMN, EPI, ACT>(P, pr, products, s);
  if constexpr (EPI != kEpiGate) {
    if (tiles(128, 128) < sms) return gemm_launch<1, 64, 1, AMN, BMN, EPI, ACT>(P, pr, products, s);
  }
  return gemm_launch<1, 128, 1, AMN, BMN, EPI, ACT>(P, pr, products, s);
}

}  // namespace prism
