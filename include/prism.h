/*
 * prism.h — C ABI of the Prism dynamic block-sparse attention hot path for
 * NVIDIA B200 (sm_100a).
 *
 * Prism ("Prism: Dynamic Sparse Attention for Native 2K Joint Video-Audio
 * Generation Model Training"; README of Tencent-Hunyuan/Prism, section
 * "Overview") organises the video token grid into spatiotemporal macro-zones,
 * gives every zone one 64-token block shape chosen from the video features'
 * channel variance and the norm of the audio-to-video (a2v) bridge residual,
 * represents blocks by block-level (mean-pooled) features, selects key blocks
 * per query block with a hybrid top-k + cumulative-mass rule, and runs exact
 * attention over the selected blocks only, forward and backward.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Token order is raster over the latent grid (T, H, W):
 *   token n = (t * H + h) * W + w.
 * - Zones tile the grid in raster (zt, zh, zw) order; zone z covers
 *   [zt*Zt, zt*Zt+Zt) x [zh*Zh, ...) x [zw*Zw, ...).
 * - A block shape is (bt, bh, bw) with bt*bh*bw == 64 dividing the zone
 *   extents. The blocks of zone z are numbered raster over the zone's
 *   (Zt/bt, Zh/bh, Zw/bw) sub-grid; global block id = z * blocks_per_zone +
 *   local id, blocks_per_zone = Zt*Zh*Zw/64. Tokens inside a block are raster
 *   (t, h, w). Query and key blocks use the same partition.
 * - Grids that are not a whole number of zones (real video latents, e.g. 45
 *   latent rows at 720p; the Prism pages train at 720p, 1080p and 2K and do
 *   not say how edges are tiled; this is the library's reading): zones tile
 *   the grid rounded up to whole zones, so n_zones = prod ceil(extent/zone),
 *   and the last zone along a clipped axis covers only the grid's remainder.
 *   Block boxes tile the unclipped zone as above and keep their ids; a block's
 *   members are the slots of its box inside the grid (fewer than 64 at the
 *   edge), and a box with no member is an empty block. Zone statistics use the
 *   member tokens (lines clipped), pooling averages the members (an empty
 *   block's pooled row is NaN), the selection never keeps an empty block and
 *   leaves its row empty, and attention runs over member tokens only.
 * - Q, K, V, O, dO, dQ, dK, dV are token-major [N, heads, head_dim] with a
 *   token stride of `tok_stride` elements (>= heads*head_dim, a multiple of 8)
 *   and contiguous heads and channels.
 * - Pointers marked "device" must be device memory of the current device;
 *   "host" pointers are read (or written) before the call returns. The
 *   library never allocates or frees device memory: scratch comes from the
 *   caller's workspace `ws` of `ws_bytes` bytes (256-byte aligned), sized by
 *   prism_workspace_size(). Its first 256 bytes, the device status word, have
 *   to be zero before the first call that uses it (prism_clear_device_status on
 *   that call's stream); the rest needs no value. Work is enqueued on `stream` (a
 *   cudaStream_t; NULL is the legacy default stream) and is asynchronous unless
 *   stated.
 * - Every call validates its arguments on the host and returns a status; no
 *   exception crosses the ABI. Device-side faults are avoided by design:
 *   device waits are bounded and report PRISM_ERR_TIMEOUT, index checks
 *   report PRISM_ERR_DEVICE, through prism_check_device_status().
 * - Not re-entrant on one workspace: calls that share `ws` must be ordered on
 *   one stream.
 */
#ifndef PRISM_H_
#define PRISM_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PRISM_API __attribute__((visibility("default")))
#else
#define PRISM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PRISM_OK = 0,
  PRISM_ERR_ARG = 1,         /* NULL where a pointer is required, bad scalar */
  PRISM_ERR_SHAPE = 2,       /* grid / zone / candidate geometry invalid */
  PRISM_ERR_DTYPE = 3,       /* dtype not supported for this argument */
  PRISM_ERR_WORKSPACE = 4,   /* ws NULL, misaligned or smaller than required */
  PRISM_ERR_CAPACITY = 5,    /* col_cap smaller than the number of kept pairs */
  PRISM_ERR_CUDA = 6,        /* a CUDA runtime / driver call failed */
  PRISM_ERR_TIMEOUT = 7,     /* a bounded device wait gave up */
  PRISM_ERR_DEVICE = 8,      /* a device-side index check failed */
  PRISM_ERR_UNSUPPORTED = 9  /* size outside what the kernels implement */
} prism_status;

typedef enum { PRISM_BF16 = 0, PRISM_FP32 = 1 } prism_dtype;

typedef struct {
  int32_t t, h, w;
} prism_dim3;

/* Token-grid geometry shared by the block-level entry points.
 * grid: latent token grid (T, H, W); zone: macro-zone extents (Zt, Zh, Zw)
 * (need not divide the grid, see above), with Zt*Zh*Zw a multiple of 64 and
 * at most 512;
 * cand: host array of n_cand (1..16) candidate block shapes. */
typedef struct {
  prism_dim3 grid;
  prism_dim3 zone;
  const prism_dim3* cand;
  int32_t n_cand;
} prism_geometry;

/* Constants of the zone shape rule (see prism_zone_shapes). */
typedef struct {
  float w_audio;  /* weight of the audio term, default 1 */
  float gamma;    /* isotropy penalty, default 0.25 */
  float gate_max; /* cap G of the audio gate, default 4 */
} prism_shape_params;

/* Which call a workspace is sized for. */
typedef enum {
  PRISM_OP_ZONE_SHAPES = 0,
  PRISM_OP_BLOCK_SELECT = 1,
  PRISM_OP_BSA_FWD = 2,
  PRISM_OP_BSA_BWD = 3
} prism_op;

/* Human-readable name of a status. Never NULL. */
PRISM_API const char* prism_status_string(prism_status s);

/* Library version, major*10000 + minor*100 + patch. */
PRISM_API int32_t prism_version(void);

/* Number of zones and of blocks for a geometry (host only, no GPU work). */
PRISM_API prism_status prism_geometry_counts(const prism_geometry* geo, int32_t* n_zones, int32_t* n_blocks);

/* Workspace bytes needed by `op`. `nnz` is the number of selected
 * (query block, key block) pairs summed over heads (row_ptr[heads*n_blocks]),
 * used by PRISM_OP_BSA_BWD only. `in_dtype` is the dtype of Q/K/V (fp32
 * inputs need bf16 staging copies). Host only. */
PRISM_API prism_status prism_workspace_size(prism_op op, const prism_geometry* geo, int32_t heads, int32_t head_dim,
                                  int32_t feat_c, int32_t res_c, prism_dtype in_dtype, int64_t nnz,
                                  size_t* bytes);

/* Clears the first 256 bytes of `ws`, in the order of `stream`. */
PRISM_API prism_status prism_clear_device_status(void* ws, void* stream);

/* Reads and clears the device status word kept in `ws` (synchronises
 * `stream`). Returns PRISM_ERR_TIMEOUT or PRISM_ERR_DEVICE if a kernel that
 * used this workspace reported one, else PRISM_OK. */
PRISM_API prism_status prism_check_device_status(void* ws, void* stream);

/* For a caller that gives its workspace up after a call: adds the status word
 * of `ws` (256 bytes read, in the order of `stream`) to one that the library
 * keeps on the current device. */
PRISM_API prism_status prism_keep_device_status(const void* ws, void* stream);

/* prism_check_device_status of what was kept, over all streams, for the work
 * that `stream` is behind. ws: a free workspace of 256 bytes; cleared. */
PRISM_API prism_status prism_check_kept_status(void* ws, void* stream);

/*
 * a1 + a2 — macro-zone tiling and per-zone block shape.
 * Cites: README "Overview" (zones; video feature variance along the channel
 * and a2v feature norms; finer partitioning along axes of rapid visual change
 * and strong audio-visual coupling); walkthrough (wmrh.cn/news/72296) section
 * "桥接残差反哺稀疏注意力" (per-token L2 norm of the unscaled a2v residual as
 * the audio-influence proxy; sounding regions get finer blocks) and section
 * "三者如何协同" (candidate shapes, one per zone).
 *
 * The rule (no formula is printed; this is the library's documented
 * reading): for zone z and axis a in (t, h, w), V_a = mean over channels and
 * over lines parallel to a of the population variance of the feature along
 * the line; r(n) = ||res[n, :]||_2, A_a = mean over lines parallel to a of
 * the population variance of r; g = clamp(mean_z r / mean_grid r - 1, 0,
 * gate_max); S_a = 3 V_a / (sum V + 1e-12) + w_audio * g * 3 A_a / (sum A +
 * 1e-12), renormalised to sum 3 (all ones when zero); cost(c) = sum_a S_a *
 * log2(ext_{c,a}) + gamma * sum_a (log2(ext_{c,a}) - 2)^2; the zone takes the
 * argmin, ties to the lower candidate index.
 *
 * feat: device [N, feat_c] row stride feat_ld elements (bf16 or fp32), or
 *       NULL; res: device [N, res_c] row stride res_ld, or NULL. Both NULL:
 *       every zone takes candidate 0. Row strides are multiples of 8 elements
 *       and feat_c / res_c multiples of 64.
 * params: host, NULL for the defaults.
 * zone_shape: device int32 [n_zones] out (candidate index per zone).
 * zone_margin: device float [n_zones] out (second-best minus best cost), or
 *       NULL.
 * A statistics kernel whose bounded wait for its copies ran out leaves every
 * zone_shape entry -1 (and every margin NaN) besides setting PRISM_ERR_TIMEOUT
 * in the workspace status word.
 */
PRISM_API prism_status prism_zone_shapes(const prism_geometry* geo, const void* feat, int64_t feat_ld, int32_t feat_c,
                               prism_dtype feat_dtype, const void* res, int64_t res_ld, int32_t res_c,
                               prism_dtype res_dtype, const prism_shape_params* params, int32_t* zone_shape,
                               float* zone_margin, void* ws, size_t ws_bytes, void* stream);

/*
 * prism_zone_shapes without a workspace (the Prism pages have no counterpart
 * to this entry point; it is a deployment variant of a1 + a2).
 *
 * For callers that cannot allocate device memory: code that runs inside a
 * host framework owning every device allocation (a serving runtime's fixed
 * pool, a plugin interface that hands out no scratch buffer), or code that must
 * not call cudaMalloc after start-up because it would synchronise the device
 * in the middle of its work. Inputs, outputs and the result are exactly those
 * of prism_zone_shapes; only the scratch differs: it lives in one static
 * device array of 4 MiB inside the library, which every GPU that loads the
 * library holds until the process exits. That bounds the grid: about 7 bytes
 * per token plus 32 per zone with 3072 bf16 channels (the 2K grid of 294,912
 * tokens needs 2.1 MB); a call that needs more returns PRISM_ERR_UNSUPPORTED.
 * The call allocates nothing (no cudaMalloc, cudaFree or allocating library
 * routine). The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress with that device current), and looks it up again when
 * the device's context has changed (after cudaDeviceReset the module is
 * reloaded and the array may move); make that first call before any stream
 * capture. All calls share the array and it keeps the last call's contents, so
 * calls that overlap on the GPU (different streams, or several host threads)
 * race and must be serialised by the caller. There is no workspace status word
 * to read back: a device-side wait that ran out shows as zone_shape entries of
 * -1 (margins NaN), which the downstream entry points reject as out of range.
 */
PRISM_API prism_status prism_zone_shapes_static(const prism_geometry* geo, const void* feat, int64_t feat_ld,
                                                int32_t feat_c, prism_dtype feat_dtype, const void* res,
                                                int64_t res_ld, int32_t res_c, prism_dtype res_dtype,
                                                const prism_shape_params* params, int32_t* zone_shape,
                                                float* zone_margin, void* stream);

/*
 * a3 — block partition and mean pooling ("block-level features", README
 * "Overview"): q_pool[h, b, :] = mean of the 64 rows Q[n, h, :] of block b,
 * likewise k_pool.
 * zone_shape: device int32 [n_zones] (from prism_zone_shapes).
 * q, k: device [N, heads, head_dim], bf16 or fp32, token stride tok_stride.
 * q_pool, k_pool: device float [heads, n_blocks, head_dim] out.
 * head_dim is 64 or 128; heads * head_dim <= 8192.
 * ws: workspace of at least prism_workspace_size(PRISM_OP_BLOCK_SELECT, ...)
 *       bytes; only its status word is used (an out-of-range zone_shape entry
 *       leaves that block's pooled rows as NaN and reports PRISM_ERR_DEVICE).
 */
PRISM_API prism_status prism_block_pool(const prism_geometry* geo, const int32_t* zone_shape, const void* q, const void* k,
                              prism_dtype dtype, int32_t heads, int32_t head_dim, int64_t tok_stride, float* q_pool,
                              float* k_pool, void* ws, size_t ws_bytes, void* stream);

/*
 * a4 + a5 — block scoring and hybrid selection (walkthrough section
 * "三者如何协同": the gating step takes the k highest-scoring blocks, then
 * extends along the CDF until cdf_threshold, default 0.20; README "Overview":
 * hybrid selection sets each query's sparsity; Sol-Attn abstract on the
 * Prism paper page: blocks ranked by a block proxy score).
 *
 * For head h and query block I: s_J = scale * q_pool[h,I] . k_pool[h,J] over
 * all key blocks J; p = softmax(s); blocks ranked by p descending, ties to the
 * lower J; m = max(top_k, min{m : p_(1) + ... + p_(m) >= cdf_threshold});
 * top_k >= n_blocks or cdf_threshold >= 1 keeps every block. The logits are
 * formed on the tensor cores in split tf32 precision (hi.hi + hi.lo + lo.hi,
 * relative error about 2^-20) for a round of heads at a time and held in the
 * workspace (a round of heads whose logits fit in 1 GiB) until that round's
 * selection has read them; they are not an output.
 *
 * q_pool, k_pool: device float [heads, n_blocks, head_dim]; n_blocks at most
 *       10240 and heads * n_blocks^2 below 2^31 (PRISM_ERR_UNSUPPORTED
 *       otherwise). A NaN pooled row marks an empty block (see the
 *       conventions): never kept as a key; as a query its row is empty.
 * top_k >= 1; cdf_threshold >= 0.
 * mask: device uint32 [heads, n_blocks, ceil(n_blocks/32)] out; bit (J % 32)
 *       of word J / 32 of row (h, I) is set when J is kept.
 * kept: device int32 [heads, n_blocks] out (m per row).
 * row_ptr: device int32 [heads*n_blocks + 1] out, CSR offsets over the rows
 *       taken in (h, I) order.
 * col_idx: device int32 [col_cap] out, kept J of each row ascending; NULL to
 *       skip (then col_cap is ignored).
 * total_kept: host int64 out (synchronises `stream`), or NULL. When col_idx
 *       is given and the total exceeds col_cap the call returns
 *       PRISM_ERR_CAPACITY after the sync, with col_idx untouched (this check
 *       needs total_kept != NULL; without it the fill clips at col_cap and
 *       reports PRISM_ERR_DEVICE through prism_check_device_status).
 * ws: at least prism_workspace_size(PRISM_OP_BLOCK_SELECT, geo, heads,
 *       head_dim, ...) bytes (equivalently prism_block_select_workspace_size):
 *       the status word, the tf32 halves of q_pool and k_pool (4 * heads *
 *       n_blocks * head_dim floats) and one round's logits (R * n_blocks *
 *       ceil4(n_blocks) floats, R = the heads whose logits fit in 1 GiB, at
 *       least 1).
 */
PRISM_API prism_status prism_block_select(const float* q_pool, const float* k_pool, int32_t heads, int32_t n_blocks,
                                int32_t head_dim, float scale, int32_t top_k, float cdf_threshold, uint32_t* mask,
                                int32_t* kept, int32_t* row_ptr, int32_t* col_idx, int64_t col_cap,
                                int64_t* total_kept, void* ws, size_t ws_bytes, void* stream);

/* Per-call selection settings of prism_block_select_ex. */
typedef struct {
  int32_t top_k;                   /* k of every head when head_top_k is NULL (>= 1) */
  float cdf_threshold;             /* tau of every head when head_cdf_threshold is NULL (>= 0) */
  const int32_t* head_top_k;       /* host int32 [heads] (each >= 1), or NULL */
  const float* head_cdf_threshold; /* host float [heads] (each >= 0), or NULL */
  const float* key_bias;           /* device float [n_blocks], or NULL: b_J added to s_J */
} prism_select_params;

/*
 * a4 + a5 with per-head settings and an optional key-block scoring bias.
 *
 * Per-head k and tau: the walkthrough (wmrh.cn/news/72296) section
 * "实际案例与上手参考" exposes the selection as a tunable knob
 * (BSA_SPARSITY, a top-k sparsity ratio); this entry point lets every head
 * carry its own floor k_h and mass threshold tau_h. Scoring bias: the same
 * walkthrough, section "桥接残差反哺稀疏注意力", says the per-token norm of the
 * a2v residual is read when BSA scores blocks and that sounding regions keep
 * more attention; with key_bias (e.g. from prism_block_audio_bias) the logits
 * become s_J = scale * q_pool[h,I] . k_pool[h,J] + b_J for every head before
 * the ranking and the softmax. Otherwise the rule, outputs and their layout
 * are those of prism_block_select, with k = k_h and tau = tau_h in row (h, I).
 * With head_top_k = head_cdf_threshold = key_bias = NULL the result is
 * identical to prism_block_select(top_k, cdf_threshold).
 *
 * params: host, required. Per-head arrays need heads <= 128
 *       (PRISM_ERR_UNSUPPORTED above); any k < 1 or tau < 0 (or NaN) returns
 *       PRISM_ERR_ARG before any work is enqueued. key_bias must be 4-byte
 *       aligned; a NaN entry gives its key block no mass.
 */
PRISM_API prism_status prism_block_select_ex(const float* q_pool, const float* k_pool, int32_t heads,
                                             int32_t n_blocks, int32_t head_dim, float scale,
                                             const prism_select_params* params, uint32_t* mask, int32_t* kept,
                                             int32_t* row_ptr, int32_t* col_idx, int64_t col_cap,
                                             int64_t* total_kept, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of prism_block_select / prism_block_select_ex for pooled
 * features of `heads` x `n_blocks` x `head_dim` (the same value as
 * prism_workspace_size(PRISM_OP_BLOCK_SELECT, ...) for that geometry's block
 * count), for callers that hold only the pooled shapes. Host only. */
PRISM_API prism_status prism_block_select_workspace_size(int32_t heads, int32_t n_blocks, int32_t head_dim,
                                                         size_t* bytes);

/*
 * Top-k floor from a top-k sparsity ratio (walkthrough section
 * "实际案例与上手参考": BSA_SPARSITY sets the top-k sparsity ratio). The library's
 * reading: the ratio is the fraction of key blocks the top-k part drops, so
 * k = n_blocks - floor(sparsity * n_blocks) with the product formed in double
 * from the float argument, at least 1; that is the smallest count that keeps
 * at least the fraction 1 - sparsity of the blocks. Host only.
 * sparsity in [0, 1), n_blocks >= 1, top_k: host out. PRISM_ERR_ARG otherwise.
 */
PRISM_API prism_status prism_topk_from_sparsity(float sparsity, int32_t n_blocks, int32_t* top_k);

/*
 * Audio-norm bias of every key block, for prism_block_select_ex (walkthrough
 * section "桥接残差反哺稀疏注意力": the per-token L2 norm of the unscaled a2v
 * residual is the proxy of how strongly audio drives a visual region, read
 * when BSA scores blocks; sounding regions keep more attention). The library's
 * reading: b_J = beta * mean_{n in block J} r(n) / mean_{all n} r(n),
 * r(n) = ||res[n, :]||_2 (fp32 per token, fp64 grid mean). The ratio makes
 * the bias independent of the residual's scale; a zero residual gives b = 0.
 *
 * zone_shape: device int32 [n_zones] (from prism_zone_shapes); the blocks are
 *       those of prism_block_pool.
 * res: device [N, res_c] (bf16 or fp32), row stride res_ld elements (a
 *       multiple of 8), res_c a positive multiple of 8, 16-byte aligned.
 * beta: finite scale of the bias (0 gives b = 0).
 * key_bias: device float [n_blocks] out.
 * ws: at least prism_workspace_size(PRISM_OP_BLOCK_SELECT, ...) bytes; only
 *       its status word is used (an out-of-range zone_shape entry leaves the
 *       whole bias NaN and reports PRISM_ERR_DEVICE).
 */
PRISM_API prism_status prism_block_audio_bias(const prism_geometry* geo, const int32_t* zone_shape, const void* res,
                                              int64_t res_ld, int32_t res_c, prism_dtype res_dtype, float beta,
                                              float* key_bias, void* ws, size_t ws_bytes, void* stream);

/*
 * Expands a selection bitmask (as written by prism_block_select) into the
 * CSR column lists: col_idx[row_ptr[r] .. row_ptr[r+1]) = the set bits of row
 * r, ascending. Use it after a prism_block_select call made with
 * col_idx = NULL and total_kept to size col_idx. Rows past col_cap are left
 * unwritten and reported through prism_check_device_status.
 * mask: device uint32 [rows, ceil(n_blocks/32)]; row_ptr: device int32
 * [rows+1]; col_idx: device int32 [col_cap] out.
 */
PRISM_API prism_status prism_mask_to_csr(const uint32_t* mask, const int32_t* row_ptr, int32_t rows, int32_t n_blocks,
                                         int32_t* col_idx, int64_t col_cap, void* ws, size_t ws_bytes, void* stream);

/*
 * a6 — block-sparse attention forward (Sol-Attn abstract: compute only the
 * selected key/value blocks): for every query token i of block I,
 * O_i = sum over key tokens j of the blocks in row (h, I) of the CSR of
 * softmax_j(scale * q_i . k_j) v_j, and lse[h, i] = log sum_j exp(scale q_i.k_j)
 * (natural log). Exact up to bf16 operand rounding; fp32 accumulation.
 *
 * zone_shape: device int32 [n_zones].
 * q, k, v: device [N, heads, head_dim], bf16 (fp32 inputs are rounded to bf16
 *       in the workspace), token stride tok_stride. head_dim 64 or 128.
 * row_ptr, col_idx: device CSR from prism_block_select (rows with no block
 *       give O = 0 and lse = -inf).
 * nnz: row_ptr[heads*n_blocks] (the total_kept of prism_block_select), or -1
 *       when the caller does not know it. It only chooses how the work is
 *       laid out: with at most 32 selected key blocks per row on average the
 *       kernel gathers K and V straight from k and v, row after row, and the
 *       workspace's block images go unused; otherwise (and for -1) K and V
 *       are first made block images. Any value >= -1 gives the same result;
 *       below -1 is PRISM_ERR_ARG.
 * o: device [N, heads, head_dim] out, same dtype as q, token stride tok_stride.
 * lse: device float [heads, N] out.
 * o_lo: optional device bf16 [N, heads, head_dim] out (token stride
 *       tok_stride), or NULL: the rounding residual of the bf16 output,
 *       O_fp32 - bf16(O_fp32), so that O_fp32 = o + o_lo to about 16 bits.
 *       Passing it to prism_bsa_bwd makes D_i = dO_i . O_i exact to that
 *       precision; with a nearly one-hot softmax, dS = P (dP - D) cancels
 *       and bf16 rounding of O alone would dominate dQ and dK. Ignored (may be
 *       NULL) for fp32 outputs, which carry no rounding.
 * ws: at least prism_workspace_size(PRISM_OP_BSA_FWD, ...) bytes. It holds
 *       block-major copies of K and V (2 * heads * n_blocks * head_dim * 128
 *       bytes: each 64-token block of each head as one contiguous, already
 *       swizzled operand tile, so the kernel gathers a key block with one bulk
 *       copy) and, for fp32 inputs, the bf16 copies of Q, K and V.
 */
PRISM_API prism_status prism_bsa_fwd(const prism_geometry* geo, const int32_t* zone_shape, const void* q, const void* k,
                           const void* v, prism_dtype dtype, int32_t heads, int32_t head_dim, int64_t tok_stride,
                           float scale, const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz, void* o,
                           float* lse, void* o_lo, void* ws, size_t ws_bytes, void* stream);

/*
 * a7 — block-sparse attention backward (Prism trains natively with the
 * sparse attention, README "Overview"), selection held fixed:
 * D_i = sum_c dO_ic O_ic; P_ij = exp(scale q_i.k_j - lse_i) on the selected
 * blocks; dV_j = sum_i P_ij dO_i; dS_ij = P_ij (dO_i . v_j - D_i);
 * dQ_i = scale sum_j dS_ij k_j; dK_j = scale sum_i dS_ij q_i.
 * Arguments as prism_bsa_fwd; o, o_lo (or NULL) and lse are the forward's
 * outputs (with o_lo, D_i = dO_i . (O_i + O_lo_i)); dout is device
 * [N, heads, head_dim]; dq, dk, dv are device outs like q. nnz =
 * row_ptr[heads*n_blocks] (for workspace sizing; checked against ws_bytes).
 * With at most 32 selected key blocks per row on average the passes gather
 * their streamed blocks straight from the inputs and the block-major copies
 * below go unused; the result is the same.
 * ws: at least prism_workspace_size(PRISM_OP_BSA_BWD, ...) bytes: D and the
 *       LSE in block order, the CSC of the selection (4 bytes per selected
 *       pair), two block-major operand copies (2 * heads * n_blocks *
 *       head_dim * 128 bytes; K and V for the dQ pass, then Q and dO for the
 *       dK/dV pass) and, for fp32 inputs, bf16 copies of Q, K, V and dO.
 */
PRISM_API prism_status prism_bsa_bwd(const prism_geometry* geo, const int32_t* zone_shape, const void* q, const void* k,
                           const void* v, const void* o, const void* o_lo, const float* lse, const void* dout,
                           prism_dtype dtype,
                           int32_t heads, int32_t head_dim, int64_t tok_stride, float scale, const int32_t* row_ptr,
                           const int32_t* col_idx, int64_t nnz, void* dq, void* dk, void* dv, void* ws,
                           size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The operators around the attention in one layer's training step: the
 * rotation of Q and K before it, the feed-forward block after it, and the
 * clipping of the gradients that the backward passes leave.
 * ---------------------------------------------------------------------- */

/* Which channels of a head form pair i of its rot_dim rotated channels. */
typedef enum {
  PRISM_ROPE_INTERLEAVED = 0, /* 2i and 2i + 1 */
  PRISM_ROPE_HALF = 1         /* i and i + rot_dim / 2 */
} prism_rope_layout;

/* How the frequencies are stretched for contexts longer than those trained. */
typedef enum {
  PRISM_ROPE_UNSCALED = 0,
  PRISM_ROPE_LINEAR = 1, /* every frequency divided by factor */
  PRISM_ROPE_NTK = 2,    /* theta * factor^(n / (n - 2)), n the axis's channels */
  PRISM_ROPE_YARN = 3    /* per pair: kept, divided by factor, or a share of both */
} prism_rope_scaling;

/*
 * The rotation. The first rot_dim = sum of axis_dim channels of a head are
 * rotated, in pairs: those of axis 0 first, then axis 1, then axis 2 (in the
 * half layout the pairs are numbered over the whole rotated part, so an axis
 * owns one run of channels in either half). Pair j of an axis of n channels
 * has the frequency theta^(-2j/n), stretched as `scaling` says; the token at
 * position p of that axis turns by (pos_offset + p * pos_scale) * frequency.
 * With PRISM_ROPE_YARN a pair that turns more than 32 times over trained_len
 * positions keeps its frequency, one that turns less than once has it divided
 * by factor, and a linear ramp over the pair's index lies between the two
 * (from floor to ceil of the border indices).
 */
typedef struct {
  int32_t layout;      /* prism_rope_layout */
  int32_t scaling;     /* prism_rope_scaling */
  int32_t n_axes;      /* 3: (t, h, w) of the token grid; 1: one position */
  int32_t axis_dim[3]; /* rotated channels of each axis, even, >= 0; their sum in 2..head_dim */
  double theta;        /* > 1 */
  double factor;       /* > 0, read unless PRISM_ROPE_UNSCALED */
  double trained_len;  /* > 0, read with PRISM_ROPE_YARN */
  double magnitude;    /* every rotated channel is multiplied by it (1: a pure rotation) */
  double pos_scale[3], pos_offset[3];
} prism_rope_params;

/*
 * Rotary positions of q and, unless k is NULL, of k.
 *
 * Pair (x1, x2) at angle a becomes m (x1 cos a - x2 sin a), m (x2 cos a + x1
 * sin a); with `transposed` the angle is -a, which is the gradient of the
 * rotation: pass dQ and dK of prism_bsa_bwd. Channels behind rot_dim keep
 * their bits. Angles are formed in 64 bits, the products in 32, and each
 * output is rounded once.
 *
 * positions: device int32 [n_tokens, n_axes], any values; NULL takes the
 *       raster order: (t, h, w) of `grid` with n_axes 3 (t * h * w ==
 *       n_tokens, PRISM_ERR_SHAPE otherwise), the token's index with 1.
 * grid: host, read only for that; may be NULL otherwise.
 * n_tokens: 0 .. 2^30; 0 does nothing.
 * q: device [n_tokens, heads_q, head_dim], k: [n_tokens, heads_k, head_dim]
 *       (heads_k may differ: grouped heads), bf16 or fp32, contiguous heads
 *       and channels, token strides in elements at least heads * head_dim and
 *       at most 2^31. head_dim is even and at most 256. Any address and stride of whole
 *       elements is taken; 16-byte alignment is fastest.
 * q_out, k_out: device outs of the same dtype, with strides of their own. An
 *       output may be exactly its input (in place); otherwise no output may
 *       share memory with another tensor of the call (PRISM_ERR_ARG; views of
 *       one packed buffer with equal strides are told apart).
 * No workspace.
 */
PRISM_API prism_status prism_rope(const prism_rope_params* params, const prism_dim3* grid, const int32_t* positions,
                                  int64_t n_tokens, const void* q, void* q_out, int32_t heads_q, int64_t q_stride,
                                  int64_t q_out_stride, const void* k, void* k_out, int32_t heads_k,
                                  int64_t k_stride, int64_t k_out_stride, prism_dtype dtype, int32_t head_dim,
                                  int32_t transposed, void* stream);

typedef enum { PRISM_NORM_L2 = 0, PRISM_NORM_INF = 1 } prism_norm_order;

/* One gradient of a list. */
typedef struct {
  void* data;     /* device, numel contiguous values; NULL allowed when numel is 0 */
  void* out;      /* where its scaled values go; NULL: in place. Not read by prism_grad_norm */
  int64_t numel;  /* >= 0 */
  int32_t dtype;  /* prism_dtype, of data and out */
  int32_t reserved;
} prism_tensor;

/*
 * Global norm over every value of a list of tensors (types may be mixed):
 * norm = sqrt(sum g^2), or the largest |g| with PRISM_NORM_INF. Sums are kept
 * in fp64 and added in a fixed order (the same bits every time for the same
 * list on the same GPU model). A NaN or infinite value shows in the norm; an
 * empty list has norm 0.
 *
 * grads: host array of n_tensors (0 .. 2^20) entries; a tensor listed twice
 *       counts twice. norm: device float out.
 * ws: at least prism_grad_norm_workspace_size(n_tensors) bytes. Norm and
 *       workspace share no memory with each other or a tensor (PRISM_ERR_ARG).
 * A step whose gradients are split over ranks (a layer sharded by heads) adds
 * up norm^2 over the ranks between prism_grad_norm and prism_grad_scale.
 */
PRISM_API prism_status prism_grad_norm(const prism_tensor* grads, int64_t n_tensors, int32_t ord, float* norm,
                                       void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of prism_grad_norm and prism_grad_clip. Host only. */
PRISM_API prism_status prism_grad_norm_workspace_size(int64_t n_tensors, size_t* bytes);

/*
 * Scales every value by min(1, max_norm / (norm + eps)) with the norm read
 * from device memory (rounded once to its type). A factor of 1 leaves in-place
 * tensors untouched; a NaN norm makes every value NaN, an infinite one makes
 * finite values 0. max_norm >= 0 (infinity: the factor is 1 whatever the norm);
 * eps >= 0 (with norm + eps = 0 the factor is 1). No tensor's output may share memory with the norm, with another
 * tensor of the list or, other than exactly, with its own input (PRISM_ERR_ARG).
 */
PRISM_API prism_status prism_grad_scale(const prism_tensor* grads, int64_t n_tensors, const float* norm,
                                        float max_norm, float eps, void* stream);

/* prism_grad_norm followed by prism_grad_scale with that norm, in fewer
 * launches and with the factor from the unrounded fp64 norm. */
PRISM_API prism_status prism_grad_clip(const prism_tensor* grads, int64_t n_tensors, int32_t ord, float max_norm,
                                       float eps, float* norm, void* ws, size_t ws_bytes, void* stream);

typedef enum {
  PRISM_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
  PRISM_ACT_GELU = 1,      /* g Phi(g) */
  PRISM_ACT_GELU_TANH = 2, /* 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) */
  PRISM_ACT_RELU = 3
} prism_activation;

/* The weights of a gated feed-forward block of model width d and inner width
 * f: device bf16 w_gate, w_up [f, d] and w_down [d, f], each with a row stride
 * in elements (w_gate and w_up may be the halves of one [2 f, d] matrix). */
typedef struct {
  const void *w_gate, *w_up, *w_down;
  int64_t gate_stride, up_stride, down_stride;
  int32_t d, f;
} prism_ffn_weights;

/*
 * Gated feed-forward block: y = (act(x w_gate^T) * (x w_up^T)) w_down^T.
 *
 * m tokens (0 .. 2^30; 0 does nothing); d and f multiples of 8, at most 2^20
 *       (PRISM_ERR_UNSUPPORTED otherwise); bf16 only (PRISM_ERR_DTYPE). Every
 *       pointer is 16-byte aligned and every row stride a multiple of 8
 *       elements, at least its row's width and below 2^31.
 * x, y: device [m, d].
 * gate, up: device [m, f] contiguous outs, or both NULL: the projections
 *       x w_gate^T and x w_up^T, rounded, for the backward pass.
 * Products accumulate in fp32; h = act(gate) * up is formed from the unrounded
 * projections and rounded to bf16 once, as an operand of the second product (of
 * at most 32 tokens it is kept to 16 bits and more, as two operands: an infinite
 * weight or input may then give NaN where one operand gives an infinity).
 * No output may share memory with gate, up or the weights, and no tensor with
 * the workspace (PRISM_ERR_ARG); y may be x.
 * ws: at least prism_gated_ffn_workspace_size(m, f, 0) bytes (the status word
 *       and h).
 */
PRISM_API prism_status prism_gated_ffn_fwd(const prism_ffn_weights* w, int64_t m, int32_t act, prism_dtype dtype,
                                           const void* x, int64_t x_stride, void* y, int64_t y_stride, void* gate,
                                           void* up, void* ws, size_t ws_bytes, void* stream);

/*
 * Gradient of prism_gated_ffn_fwd at the saved projections gate, up [m, f]
 * (contiguous): with dh = dy w_down, dg = dh up act'(gate), du = dh act(gate)
 * (each rounded to bf16 once, or of at most 32 tokens kept to 16 bits and more):
 * dx = dg w_gate + du w_up, dw_gate = dg^T x, dw_up = du^T x,
 * dw_down = dy^T (act(gate) up). relu'(0) = 0.
 * dx: device [m, d] out, or NULL. dw_gate, dw_up [f, d], dw_down [d, f]: device
 *       contiguous outs, or all NULL (frozen weights). m = 0 zeroes them.
 * No output may share memory with any other tensor of the call, and none with
 * the workspace (PRISM_ERR_ARG).
 * ws: at least prism_gated_ffn_workspace_size(m, f, 1) bytes (the status word,
 *       dg, du and act(gate) up).
 */
PRISM_API prism_status prism_gated_ffn_bwd(const prism_ffn_weights* w, int64_t m, int32_t act, prism_dtype dtype,
                                           const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                           const void* gate, const void* up, void* dx, int64_t dx_stride,
                                           void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                           void* stream);

/* Host only, for tests and tuning: the kernel of each product of such a call of
 * m tokens with contiguous rows. forms: host int32[9] out, three values each
 * for the gate and the down product (backward 0), or for the gradient of the
 * gate, dx and the weight gradients (1): CTAs that share a tile (1, or a pair),
 * its accumulator's columns (0: the persistent kernel of pairs) and the parts
 * of K that a cluster splits it into; all 0: no such product, or the kernel of
 * a handful of tokens. */
PRISM_API prism_status prism_gated_ffn_forms(const prism_ffn_weights* w, int64_t m, int32_t backward, int32_t* forms);

/* Workspace bytes of prism_gated_ffn_fwd (backward 0) and _bwd (1). Host only. */
PRISM_API prism_status prism_gated_ffn_workspace_size(int64_t m, int32_t f, int32_t backward, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* PRISM_H_ */
