// The matrix product of gemm.cuh for few tiles: a cluster shares one tile (128 x
// BN of single CTAs, 256 x BN of pairs), each CTA or pair multiplying its part
// of K; the partial sums meet in distributed shared memory.
//
// With few tokens or a small layer there are fewer tiles than SMs, and an SM
// fetches at most some 90 GB/s from L2 (measured), so a product is as fast as
// its operands' bytes are spread over SMs. Splitting K needs the sums of the
// parts: every CTA leaves its fp32 partial tile in its own shared memory (where
// the operand slices were), and after a cluster barrier sends row part r of it to
// part r of the CTAs in one bulk copy (loads of the other CTAs' shared memory
// took 3 to 4 us for the same, 128 x 128 in 4 parts); that one adds what it got in
// the order of the parts (the same bits every time, no atomics, no workspace) and
// applies the epilogue. Of an operand
// A with fewer than 128 rows only those (rounded up to 8) are copied: the tensor
// cores read stale rows beyond them, whose sums nobody reads.
// A copy comes back after about 1.5 us, so the ring holds as many slices as
// shared memory takes: all of it when there is a CTA per SM at most, else half,
// for two CTAs per SM, one's epilogue beside the other's copies.
#pragma once
#include "gemm.cuh"

namespace prism {

constexpr int kSplitMax = 8;      // CTAs of a cluster
constexpr int kSplitStages = 16;  // most slices of a ring

struct SplitArgs {
  CUtensorMap a[2], b[2];  // as in GemmProduct
  const __nv_bfloat16* in[2];  // kEpiGateBwd: the saved projections [m, n], contiguous
  __nv_bfloat16* out[3];
  int64_t out_ld[3];
  int m, n;
  int tiles_m, tiles_n, tile0;
  int slices0, slices;
};

struct SplitLaunch {
  SplitArgs p[kGemmProducts];
  int products, save, beside, fine, fold;  // see GemmArgs
  int a_bytes, stages;  // of A's part of a slice, and slices of the ring
  int slot_rows;        // rows of a part's share of another CTA's rows, at most
  int* status;
};

// Shared memory: barriers (1 KB), then the ring. The tensor cores read 16 KB
// from the start of a slice's A, whatever was copied, so the last slice is
// followed by room for that. The fp32 partial tile and what the other parts send
// take the ring's place.
constexpr int kSplitBars = 1024;
constexpr int split_pitch(int bn) { return bn + 4; }  // floats between its rows: 16 bytes modulo 32 banks apart
constexpr int split_tile_rows(int a_bytes) { return (a_bytes / 128 + 31) / 32 * 32; }  // a warp's 32 rows at a time
constexpr int split_smem(int cg, int bn, int a_bytes, int stages, int parts, int slot_rows) {
  const int ring = stages * (a_bytes + bn / cg * 128) + kGemmM * 128 - a_bytes;
  const int tile = (split_tile_rows(a_bytes) + (parts - 1) * slot_rows) * split_pitch(bn) * 4;
  return 1024 + kSplitBars + (ring > tile ? ring : tile);
}

// `bytes` (a multiple of 16) of this CTA's shared memory to another of its
// cluster, counted on that one's barrier.
__device__ __forceinline__ void bulk_send(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// The sum over the parts, in their order, of 8 values: this CTA's at `own`, part
// p's at `got` + (p or, behind this CTA's, p - 1) * slot.
__device__ __forceinline__ void sum_parts(const float* own, const float* got, int slot, int parts, int part_of, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int p = 0; p < parts; ++p) {
    const float* a = p == part_of ? own : got;
    if (p != part_of) got += slot;
    const float4 x = *reinterpret_cast<const float4*>(a), y = *reinterpret_cast<const float4*>(a + 4);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// 8 values to `to`, rounded, and with `fine` their remainders `below` elements further on.
__device__ __forceinline__ void store8(__nv_bfloat16* to, const float* v, bool fine, int64_t below) {
  const uint4 h = pack8(v);
  *reinterpret_cast<uint4*>(to) = h;
  if (fine) {
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r[i] = remainder_bf16(v[i], __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16));
    *reinterpret_cast<uint4*>(to + below) = pack8(r);
  }
}
__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int CG, int BN, bool AMN, bool BMN, int EPI, int ACT>
__global__ void __launch_bounds__(kGemmThreads, CG == 2 ? 1 : 2) gemm_split_kernel(const __grid_constant__ SplitLaunch P) {
  constexpr int kPitch = split_pitch(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm);
  uint64_t* empty = full + kSplitStages;
  uint64_t* acc_full = empty + kSplitStages;
  uint64_t* joined = acc_full + 1;  // the other parts' rows have come
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), cta = CG == 2 ? rank & 1 : 0, leader = rank - cta;
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int part_of = int(rank) / CG, parts = int(ranks) / CG;  // of K
  int t = blockIdx.x / ranks, prod = 0;
  while (prod + 1 < P.products && t >= P.p[prod + 1].tile0) ++prod;
  const SplitArgs& Q = P.p[prod];
  t -= Q.tile0;
  constexpr int kCols = EPI == kEpiGate ? BN / 2 : BN;  // output columns
  const int row0 = ((t % Q.tiles_m) * CG + int(cta)) * kGemmM, tn = t / Q.tiles_m, col0 = tn * kCols;
  const int first = int(int64_t(Q.slices) * part_of / parts), last = int(int64_t(Q.slices) * (part_of + 1) / parts);
  int* status = P.status;
  sm += kSplitBars;
  const int stages = P.stages, stage_bytes = P.a_bytes + BN / CG * 128;
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&Q.a[0]);
    tma_prefetch_desc(&Q.b[0]);
    if (EPI == kEpiGate) tma_prefetch_desc(&Q.b[1]);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(joined, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  auto copy = [&](int kc, int st) {
    const int seg = kc >= Q.slices0;
    const int k0 = (kc - (seg ? Q.slices0 : 0)) * kGemmK;
    const uint32_t dst = smem_u32(sm + st * stage_bytes);
    uint32_t bar = smem_u32(&full[st]);
    if constexpr (CG == 2) bar = map_shared(bar, leader);
    if (cta == 0) mbar_arrive_expect_tx(&full[st], CG * stage_bytes);
    gemm_load<CG, AMN>(dst, &Q.a[seg], bar, row0, k0, kGemmM);
    if constexpr (EPI == kEpiGate && CG == 2) {
      gemm_load<CG, BMN>(dst + P.a_bytes, &Q.b[cta], bar, col0, k0, BN / 2);
    } else if constexpr (EPI == kEpiGate) {
      gemm_load<CG, BMN>(dst + P.a_bytes, &Q.b[0], bar, col0, k0, BN / 2);
      gemm_load<CG, BMN>(dst + P.a_bytes + BN / 2 * 128, &Q.b[1], bar, col0, k0, BN / 2);
    } else {
      gemm_load<CG, BMN>(dst + P.a_bytes, &Q.b[seg], bar, col0 + int(cta) * (BN / CG), k0, BN / CG);
    }
  };
  // a ring of fresh slices needs nothing of the others' setup (of a pair, the other CTA's barriers)
  const int ahead = CG == 2 ? 0 : min(stages, last - first);
  if (threadIdx.x == 0 && ahead > 0) {
    if (!P.beside) grid_dependency_wait();
    for (int i = 0; i < ahead; ++i) copy(first + i, i);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, BN);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (!P.beside) grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int st = ahead == stages ? 0 : ahead, issued = ahead;
      uint32_t phase = ahead == stages ? 0 : 1;  // of `empty`: a fresh barrier passes
      for (int kc = first + ahead; kc < last; ++kc, ++issued) {
        ok = mbar_wait_abortable(&empty[st], phase, status, abort_flag);
        if (!ok) break;
        copy(kc, st);
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
      }
      // the leader's barriers count both CTAs' copies
      if (cta == 0)
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
          mbar_wait(&full[i % stages], (i / stages) & 1, status);
    }
  } else if (warp == 1) {
    if (lane == 0 && cta == 0) {
      const uint32_t idesc = idesc_bf16_f32(kGemmM * CG, BN, AMN, BMN);
      constexpr uint64_t kStepA = (AMN ? 2048 : 32) >> 4, kStepB = (BMN ? 2048 : 32) >> 4;
      bool ok = true;
      int st = 0;
      uint32_t phase = 0;
      for (int kc = first; kc < last; ++kc) {
        ok = mbar_wait_abortable(&full[st], phase, status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(sm + st * stage_bytes);
        const uint64_t da = sdesc_sw128(sa, AMN ? 8192 : 16, 1024);
        const uint64_t db = sdesc_sw128(sa + P.a_bytes, BMN ? 8192 : 16, 1024);
#pragma unroll
        for (int k = 0; k < kGemmK / 16; ++k)
          mma_bf16<CG>(tbase, da + k * kStepA, db + k * kStepB, idesc, (kc > first || k > 0) ? 1u : 0u);
        mma_commit_all<CG>(&empty[st], leader);
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
      }
      mma_commit_all<CG>(acc_full, leader);
    }
    // also in the pair's other CTA, which issues nothing
    if (lane == 0) mbar_wait_abortable(acc_full, 0, status, abort_flag);
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
  // the rows of the tile that this CTA finishes, 8 columns of a row per thread and step (n is a multiple of 8)
  const int rows = min(kGemmM, Q.m - row0), vecs = (min(kCols, Q.n - col0) + 7) / 8;
  const int rows_out = EPI == kEpiStore && P.fold ? P.fold : rows;
  auto row_part = [&](int p) { return rows_out * p / parts; };
  const int r0 = row_part(part_of), mine = row_part(part_of + 1) - r0, items = mine * (kCols / 8);
  uint4 gv = make_uint4(0, 0, 0, 0), uv = gv;
  auto fetch = [&](int x) {  // the saved projections of step x
    const int v = x % (kCols / 8);
    if (x >= items || v >= vecs) return;
    const int64_t at = int64_t(row0 + r0 + x / (kCols / 8)) * Q.n + col0 + 8 * v;
    gv = __ldg(reinterpret_cast<const uint4*>(Q.in[0] + at));
    uv = __ldg(reinterpret_cast<const uint4*>(Q.in[1] + at));
  };
  if constexpr (EPI == kEpiGateBwd) fetch(threadIdx.x);
  // every copy has landed and every product is complete: the slices' place is free
  __syncthreads();
  tc_fence_after();
  const bool gave_up = *abort_flag;
  float* part = reinterpret_cast<float*>(sm);
  float* got = part + split_tile_rows(P.a_bytes) * kPitch;
  if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    if (32 * q < rows) {
      float* to = part + (32 * q + lane) * kPitch;
#pragma unroll
      for (int c = half * 32; c < BN; c += 64) {
        uint32_t r[32];
        tmem_ld32(tbase + (uint32_t(q * 32) << 16) + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(to + c + 4 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      }
    }
  }
  if (parts > 1) fence_proxy_async_smem();
  __syncwarp();
  tc_fence_before();
  if (ranks == 1) __syncthreads();
  else cluster_sync_all();
  if (parts > 1) {
    const int folds = EPI == kEpiStore && P.fold ? 2 : 1;  // runs of rows that a part sends to another
    if (threadIdx.x == 0 && mine > 0) mbar_arrive_expect_tx(joined, (parts - 1) * folds * mine * kPitch * 4);
    if (warp == 0 && lane < parts && lane != part_of) {
      const int to0 = row_part(lane), n = row_part(lane + 1) - to0;
      const uint32_t to = CG * lane + cta, bar = map_shared(smem_u32(joined), to);
      const uint32_t dst = map_shared(smem_u32(got + (part_of - (part_of > lane)) * P.slot_rows * kPitch), to);
      if (n > 0) {
        for (int i = 0; i < folds; ++i)
          bulk_send(dst + i * n * kPitch * 4, part + (to0 + i * P.fold) * kPitch, n * kPitch * 4, bar);
      }
    }
    if (mine > 0) mbar_wait(joined, 0, status);
  }
  if (!gave_up) {
    for (int x = threadIdx.x; x < items; x += kGemmThreads) {
      const int r = r0 + x / (kCols / 8), v = x % (kCols / 8);
      if (v >= vecs) continue;
      const float *own = part + r * kPitch + 8 * v, *sent = got + (r - r0) * kPitch + 8 * v;
      const int slot = P.slot_rows * kPitch;
      const int64_t row = row0 + r;
      const int col = col0 + 8 * v;
      float d[8];
      sum_parts(own, sent, slot, parts, part_of, d);
      if constexpr (EPI == kEpiStore) {
        if (P.fold) {
          float e[8];
          sum_parts(own + P.fold * kPitch, sent + mine * kPitch, slot, parts, part_of, e);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += e[i];
        }
        *reinterpret_cast<uint4*>(Q.out[0] + row * Q.out_ld[0] + col) = pack8(d);
      } else if constexpr (EPI == kEpiGate) {
        float u[8], h[8];
        sum_parts(own + BN / 2, sent + BN / 2, slot, parts, part_of, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = act_f<ACT>(d[i]) * u[i];
        store8(Q.out[0] + row * Q.out_ld[0] + col, h, P.fine, Q.m * Q.out_ld[0]);
        if (P.save) {
          *reinterpret_cast<uint4*>(Q.out[1] + row * Q.out_ld[1] + col) = pack8(d);
          *reinterpret_cast<uint4*>(Q.out[2] + row * Q.out_ld[2] + col) = pack8(u);
        }
      } else {
        float g[8], u[8], dg[8], du[8], h[8];
        unpack8(gv, g);
        unpack8(uv, u);
        fetch(x + kGemmThreads);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float a, s;
          act_slope_f<ACT>(g[i], a, s);
          dg[i] = d[i] * u[i] * s;
          du[i] = d[i] * a;
          h[i] = a * u[i];
        }
        store8(Q.out[0] + row * Q.out_ld[0] + col, dg, P.fine, Q.m * Q.out_ld[0]);
        store8(Q.out[1] + row * Q.out_ld[1] + col, du, P.fine, Q.m * Q.out_ld[1]);
        if (P.save) store8(Q.out[2] + row * Q.out_ld[2] + col, h, P.fine, Q.m * Q.out_ld[2]);
      }
    }
  }
  __syncwarp();
  if (ranks == 1) __syncthreads();
  else cluster_sync_all();  // all that this CTA sent has come
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tbase, BN);
  }
  if (P.beside) grid_dependency_wait();
}

}  // namespace prism
