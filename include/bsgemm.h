/*
 * bsgemm.h - C ABI of the MI355X (gfx950) grouped block-scaled low-precision GEMM.
 *
 * The operation is the grouped, blockwise-FP8 MoE matmul whose per-K-block promote step is
 * described on the Modular MAX page "promote_accumulators"
 * (kernels/linalg/grouped_matmul_sm100_blockwise_fp8; description paragraph and section
 * Args), with the per-K-iteration cadence of the Modular MAX page "EpilogueWarpContext"
 * (method per_k_stage), plus the MX variant of the Triton Gluon page "Overlapping
 * Accumulator Block-Scaled Matrix Multiplication" (e8m0 scale per 32 K-elements, applied
 * inside the matrix instruction; reference result A_ref @ B_ref^T in its make_problem).
 *
 * General rules for every entry point:
 *  - Pointers marked DEVICE are device (HBM) pointers owned by the caller. The library
 *    never allocates, frees or retains them. Pointers marked HOST are host pointers.
 *  - Work is enqueued asynchronously on `stream` (a hipStream_t passed as void*; NULL means
 *    the null stream) on the current HIP device. Calls return after enqueueing.
 *  - Return value: BSG_OK (0) or a negative bsg_status. Arguments are validated on the host
 *    before anything is enqueued; on any error nothing is enqueued and outputs are untouched.
 *  - Thread-safe: no global mutable state apart from a per-device property cache.
 *  - Device-side contents (tile map, counts) cannot be checked on the host. The kernels clamp
 *    them instead: a tile whose expert id is outside [0, num_experts) is skipped, rows are
 *    clamped into [0, M), and negative counts count as zero. Such input gives unspecified
 *    (but in-bounds) results.
 */
#ifndef BSGEMM_H
#define BSGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BSG_OK = 0,
  BSG_ERR_NULL = -1,    /* a required pointer is NULL                                   */
  BSG_ERR_SHAPE = -2,   /* a size is negative, too large, or not a multiple it must be  */
  BSG_ERR_ALIGN = -3,   /* a pointer is not aligned as documented                      */
  BSG_ERR_FMT = -4,     /* unsupported fmt combination                                 */
  BSG_ERR_DEVICE = -5,  /* no HIP device, or the current device is not gfx950          */
  BSG_ERR_LAUNCH = -6   /* the HIP runtime rejected a kernel launch                    */
} bsg_status;

/* ---- fmt: element formats, scale kind and output type, packed into one word ------------ */
#define BSG_ELEM_E4M3 1u   /* OCP e4m3fn, one byte per element                            */
#define BSG_ELEM_E2M1 2u   /* OCP e2m1, two per byte along K, even K index in low nibble  */
#define BSG_SCALE_BLOCKWISE 1u /* fp32: A per row per 128 K; B per 128 (N) x 128 (K) block */
#define BSG_SCALE_MX 2u        /* e8m0 (uint8, 2^(x-127)): one per row per 32 K, A and B   */
#define BSG_SCALE_NV 3u        /* nvfp4: e4m3fn (uint8) scale per row per 16 K, A and B    */
#define BSG_OUT_F32 1u
#define BSG_OUT_BF16 2u
#define BSG_OUT_F16 3u
#define BSG_FMT(a_elem, b_elem, scale, out) \
  ((uint32_t)(a_elem) | ((uint32_t)(b_elem) << 4) | ((uint32_t)(scale) << 8) | ((uint32_t)(out) << 12))
/* Schedule hint (OR into fmt; blockwise only): M-tiles hold few rows (decode-sized expert
 * groups). Each work item is then one M-tile x 256 columns, and the matrix work stops at the
 * tile's last row of 16-row fragments, instead of a 256 x 256 block tile. Same results, bit for
 * bit (same instruction, operand roles and promotion order). Only the packed tile layout
 * (bsgemm_build_tiles with padded == 0) has tiles of fewer than 128 rows: with the padded layout
 * every tile spans 128 rows (padding included), so no fragment is skipped and the hint only
 * changes the work item's shape. */
#define BSG_SCHED_SMALL_M (1u << 16)

/*
 * bsgemm_build_tiles - token-to-expert tile map (the scheduler build).
 *
 * Passage: "promote_accumulators", section Args, argument expert_ids (maps a group of rows
 * to its expert in B) and argument scheduler (tracks the current group and work tile).
 *
 * Rows of A are grouped by expert in ascending expert order. From the per-expert row counts
 * this writes, with T = num_tiles:
 *   expert_offsets[e]  first row of expert e's group; expert_offsets[E] = rows the layout needs
 *   tile_offsets[t]    first row of M-tile t (t in [0, T]); tile t owns
 *                      min(128, max(0, tile_offsets[t+1] - tile_offsets[t])) rows
 *   expert_ids[t]      expert of M-tile t, or -1 for tiles past the last expert's rows
 * padded != 0: each group starts at a multiple of 128 rows, tile_offsets[t] = 128 t, and tiles
 *   include the group's padding rows.
 * padded == 0: groups are packed back to back; each group's last tile is ragged; tiles past
 *   the last one start at expert_offsets[E].
 * If the layout needs more than T tiles, the extra tiles are dropped (expert_offsets[E] still
 * reports the rows needed, so the caller can detect it).
 *
 *   counts          DEVICE int32[num_experts], row count per expert (>= 0)
 *   num_experts     1 .. 4096
 *   num_tiles       >= 0
 *   expert_offsets  DEVICE int32[num_experts + 1] (output)
 *   tile_offsets    DEVICE int32[num_tiles + 1]   (output)
 *   expert_ids      DEVICE int32[num_tiles]       (output; may be NULL iff num_tiles == 0)
 * Errors: BSG_ERR_NULL, BSG_ERR_SHAPE, BSG_ERR_ALIGN (int32 alignment), BSG_ERR_DEVICE,
 * BSG_ERR_LAUNCH.
 */
int bsgemm_build_tiles(const int32_t* counts, int32_t num_experts, int32_t num_tiles,
                       int32_t padded, int32_t* expert_offsets, int32_t* tile_offsets,
                       int32_t* expert_ids, void* stream);

/*
 * bsgemm_grouped - grouped block-scaled GEMM  C[rows of tile t] = A[rows] * B[e]^T, e = expert_ids[t].
 *
 * Blockwise (scale kind BSG_SCALE_BLOCKWISE; passage: "promote_accumulators", description
 * paragraph, and Args b_scales / b_scales_n / k_iter / expert_ids / problem_shape):
 *   for every K block kb of 128:  P = sum_{k in kb} qa[m,k] * qb[e,n,k]   (fp32, fresh each block)
 *                                 acc[m,n] += P * (a_scales[m,kb] * b_scales[e, n/128, kb])
 *   C[m,n] = acc[m,n] converted to the output type (round to nearest even).
 * MX (BSG_SCALE_MX; passage: Gluon page, random_quantized_tensor / async_mma_scaled_impl):
 *   C[m,n] = sum_k (qa[m,k] 2^(sa[m,k/32]-127)) (qb[e,n,k] 2^(sb[e,n,k/32]-127)), scales
 *   applied by the gfx950 scaled matrix instruction, fp32 accumulation.
 * nvfp4 (BSG_SCALE_NV; passage: Gluon page, random_quantized_tensor for "nvfp4", VEC_SIZE 16,
 *   scales converted to float8_e4m3fn):
 *   C[m,n] = sum_k (e2m1(qa[m,k]) e4m3(sa[m,k/16])) (e2m1(qb[e,n,k]) e4m3(sb[e,n,k/16])), each
 *   scaled element formed exactly in f16, fp32 accumulation.
 *
 * Layouts (all row-major, contiguous):
 *   A          DEVICE [M, K] e4m3 bytes, or [M, K/2] packed e2m1. 16-byte aligned.
 *   a_scales   blockwise: DEVICE float[M, K/128];  MX: DEVICE uint8[M, K/32]. 4-byte aligned.
 *              nvfp4: DEVICE uint8[M, K/16] e4m3fn codes, 16-byte aligned.
 *   B          DEVICE [num_experts, N, K] e4m3 (or [num_experts, N, K/2] e2m1): K contiguous,
 *              i.e. each expert's B is stored N-major ("NT" GEMM). 16-byte aligned.
 *   b_scales   blockwise: DEVICE float[num_experts, N/128, K/128];
 *              MX: DEVICE uint8[num_experts, N, K/32]. 4-byte aligned.
 *              nvfp4: DEVICE uint8[num_experts, N, K/16] e4m3fn codes, 16-byte aligned.
 *   expert_ids DEVICE int32[num_tiles] and tile_offsets DEVICE int32[num_tiles + 1], as written
 *              by bsgemm_build_tiles (either layout). Both NULL: one dense group, expert 0,
 *              tiles of 128 rows, num_tiles ignored (M need not be a multiple of 128).
 *   C          DEVICE [M, N] float / bf16 / fp16. 16-byte aligned. Rows of skipped tiles and
 *              rows no tile covers are not written.
 * Sizes: M >= 0 (M = 0 is a no-op), N > 0 and K > 0, both multiples of 128; num_experts >= 1;
 *   num_tiles >= 0.
 * Supported fmt: blockwise with A = B = e4m3, any output type (optionally | BSG_SCHED_SMALL_M);
 *   MX with A, B in {e4m3, e2m1}, any output type;
 *   nvfp4 with A = B = e2m1 and K a multiple of 256 (else BSG_ERR_SHAPE), any output type.
 * Errors: BSG_ERR_NULL, BSG_ERR_SHAPE, BSG_ERR_ALIGN, BSG_ERR_FMT, BSG_ERR_DEVICE,
 *   BSG_ERR_LAUNCH.
 */
/*
 * Arguments beyond the problem statement's list. The operation is named with the arguments
 * (A, a_scales, B, b_scales, expert_ids, tile_offsets, C, M, N, K, fmt, stream). Two more are
 * taken here: num_tiles, the length of expert_ids (a ragged, unpadded layout has a tile count
 * that M does not determine, and the kernels never read past it), and num_experts, the leading
 * dimension of B and b_scales ("promote_accumulators", Args: b_scales is shaped
 * [num_experts, N // BN, K // BK]), so that an out-of-range expert id is skipped instead of
 * addressing past B. Neither changes the result for a valid tile map.
 */
int bsgemm_grouped(const void* A, const void* a_scales, const void* B, const void* b_scales,
                   const int32_t* expert_ids, const int32_t* tile_offsets, int32_t num_tiles,
                   void* C, int32_t M, int32_t N, int32_t K, int32_t num_experts, uint32_t fmt,
                   void* stream);

/*
 * bsgemm_grouped_workspace_size - bytes of workspace bsgemm_grouped_ws needs on the current device.
 *
 *   bytes   HOST size_t* (output): 4 KiB of flags plus one 256 x 256 fp32 tile per workgroup of
 *           the split schedule (one per compute unit, rounded down to a multiple of 8: 64 MiB + 4 KiB
 *           on a 256-CU MI355X)
 * Errors: BSG_ERR_NULL, BSG_ERR_DEVICE.
 */
int bsgemm_grouped_workspace_size(size_t* bytes);

/*
 * bsgemm_grouped_ws - bsgemm_grouped with a workspace for a split-K schedule of small problems.
 *
 * Same operation, arguments and results as bsgemm_grouped (up to the rounding order of fp32 sums:
 * outputs are within the same tolerance, not bit-identical). bsgemm_grouped runs one 256 x 256
 * work item per workgroup, so a problem with fewer items than compute units leaves units idle
 * (a 256 x 2048 x 16384 GEMM has 8 items for 256 units). With a workspace, such blockwise calls
 * cut each item along K into 2-16 equal ranges of at least 8 K blocks (as many as the grid
 * holds) that run side by side: each range accumulates its K blocks as described under
 * bsgemm_grouped into an fp32 partial tile, and the item's result is the sum of its ranges'
 * partials (each range sums and stores a slice of the tile). Blockwise problems with at least as
 * many items as compute units run whole items as bsgemm_grouped does, bit for bit, with two
 * exceptions that use the workspace's first 4 KiB as counters and flags (cleared on the stream
 * before the launch):
 *  - when K is at least 5120 (40 K blocks), the workgroups take the items of each XCD from a
 *    counter instead of a fixed sequence, which keeps the items in flight on an XCD close
 *    together in the work order (same per-item arithmetic: still bit for bit);
 *  - with fewer than 4 items per compute unit, the items of the last, partial round (items modulo
 *    the grid) are cut along K into 2-16 ranges of at least 4 K blocks, which the workgroups that
 *    run out of whole items first take from a counter, summed as above; outputs of those items
 *    are within the tolerance, not bit-identical to bsgemm_grouped, and the same on every call.
 * Formats other than blockwise and the small-M hint run exactly as bsgemm_grouped and leave the
 * workspace untouched.
 *
 *   workspace        DEVICE, 256-byte aligned, at least bsgemm_grouped_workspace_size bytes,
 *                    owned by the caller; no initial contents are required (what a launch
 *                    uses of it is cleared on the stream before the launch). Its int32 word 1023 is
 *                    an error word: nonzero after a call if a range ever stopped waiting for the
 *                    other ranges of its item (not expected while the call has the GPU's compute
 *                    units to itself: the ranges wait for ranges that running workgroups have
 *                    taken; that item's output is then wrong).
 *   workspace_bytes  its size
 * Calls that share a workspace must be ordered (one stream, or synchronised): concurrent calls
 * on one workspace race.
 * Errors: as bsgemm_grouped, plus BSG_ERR_NULL (workspace NULL), BSG_ERR_ALIGN, BSG_ERR_SHAPE
 * (workspace too small).
 */
int bsgemm_grouped_ws(const void* A, const void* a_scales, const void* B, const void* b_scales,
                      const int32_t* expert_ids, const int32_t* tile_offsets, int32_t num_tiles,
                      void* C, int32_t M, int32_t N, int32_t K, int32_t num_experts, uint32_t fmt,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * bsgemm_grouped_noalloc - bsgemm_grouped_ws without a workspace argument, allocating nothing.
 *
 * For callers that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation). Same operation, arguments, results and errors as
 * bsgemm_grouped; its split-K schedule for small problems (see bsgemm_grouped_ws) uses a scratch
 * array the library holds on each device it runs on, for the life of the process: 16 MiB + 4 KiB,
 * room for 64 partial tiles. Where bsgemm_grouped_ws would cut the items into more ranges than
 * 64 tiles, fewer ranges are used, so no call needs more scratch than the array holds and none
 * is rejected for it (results are within the same tolerance). What a launch uses of the scratch
 * (the split schedule's flags, the work-order counters) is cleared on the stream before it.
 * Every call on a GPU shares that GPU's scratch: calls that overlap on one GPU (different streams
 * or host threads without ordering) race and give wrong results. No hipMalloc, hipFree or other
 * allocating call is made.
 */
int bsgemm_grouped_noalloc(const void* A, const void* a_scales, const void* B, const void* b_scales,
                           const int32_t* expert_ids, const int32_t* tile_offsets, int32_t num_tiles,
                           void* C, int32_t M, int32_t N, int32_t K, int32_t num_experts, uint32_t fmt,
                           void* stream);

/*
 * bsgemm_route_counts - picks per expert: the row counts of the grouped A.
 *
 * Passage: "promote_accumulators", section Args, argument expert_ids (each group of A's rows
 * belongs to one expert) - the counts that bsgemm_build_tiles turns into the group layout.
 *
 *   topk_ids    DEVICE int32[num_picks]: expert of each pick, usually [tokens, top_k]
 *               row-major. Ids outside [0, num_experts) are not counted.
 *   num_picks   >= 0
 *   num_experts 1 .. 4096
 *   counts      DEVICE int32[num_experts] (output; overwritten)
 * Errors: BSG_ERR_NULL, BSG_ERR_SHAPE, BSG_ERR_ALIGN (int32 alignment), BSG_ERR_DEVICE,
 * BSG_ERR_LAUNCH.
 */
int bsgemm_route_counts(const int32_t* topk_ids, int32_t num_picks, int32_t num_experts,
                        int32_t* counts, void* stream);

/*
 * bsgemm_quantize_permute - token activations and top-k picks -> the grouped GEMM's A operand.
 *
 * Passage: "promote_accumulators", section Args (A's rows grouped by expert through
 * expert_ids; an fp32 scale per row per 128 K-elements, the 1x128 block scaling of the FP8
 * operands). The pages do not order rows inside a group; here expert e's picks fill rows
 * expert_offsets[e], expert_offsets[e] + 1, ... in pick order (token-major), which makes the
 * layout unique.
 *
 *   dest[t, j]   = A row of pick (t, j), or -1 if its id is outside [0, num_experts) or the
 *                  row would be >= M
 *   per token t and 128-block b of x[t]:  s = amax / 448 (1 if amax = 0),
 *                  q = round-to-nearest-even e4m3fn of clamp(x / s, -448, 448), both divisions
 *                  in fp32; qa[dest[t, j], block b] = q and a_scales[dest[t, j], b] = s
 *   rows expert_offsets[e] + count_e .. expert_offsets[e + 1] - 1 (below M): zero codes,
 *                  scale 1 (the group's padding); all other rows of qa / a_scales untouched
 *
 *   x              DEVICE [tokens, K] fp32 or bf16 (x_dtype BSG_OUT_F32 / BSG_OUT_BF16),
 *                  finite values. 16-byte aligned.
 *   topk_ids       DEVICE int32[tokens, top_k]
 *   tokens >= 0, top_k >= 1, K > 0 a multiple of 128, num_experts 1 .. 4096
 *   expert_offsets DEVICE int32[num_experts + 1], as written by bsgemm_build_tiles from
 *                  bsgemm_route_counts' counts (padded: each group a multiple of 128 rows)
 *   M              rows of qa / a_scales (>= 0)
 *   dest           DEVICE int32[tokens, top_k] (output)
 *   qa             DEVICE uint8[M, K] e4m3fn codes (output), 16-byte aligned
 *   a_scales       DEVICE float[M, K/128] (output)
 * Errors: BSG_ERR_NULL, BSG_ERR_SHAPE, BSG_ERR_ALIGN, BSG_ERR_FMT (x_dtype), BSG_ERR_DEVICE,
 * BSG_ERR_LAUNCH.
 */
int bsgemm_quantize_permute(const void* x, uint32_t x_dtype, const int32_t* topk_ids,
                            int32_t tokens, int32_t top_k, int32_t K, int32_t num_experts,
                            const int32_t* expert_offsets, int32_t M, int32_t* dest, void* qa,
                            float* a_scales, void* stream);

/* ======================================================================================= *
 * The steps around the grouped GEMM of an MoE block: norm, sort, rows there and back,
 * activation, quantisation, and the product for a decode batch.
 *
 * Rules beyond the general ones above: row types (x_dtype, dtype) are the BSG_OUT_* codes, rows
 * are contiguous, sums and statistics are fp32, and a result in a row type is rounded once (to
 * nearest even). Outputs do not overlap inputs except where said. The same call on the same inputs
 * gives the same bits: there are no floating-point atomics. All are safe to capture into a HIP graph
 * (kernels only). NaN and infinities go through the formulas, in their own row or token only (and sums
 * over rows).
 * ======================================================================================= */

/* q_fmt: a quantised output's element type and scale kind. Supported (K a multiple of 128):
 *   (E4M3, BLOCKWISE)  codes uint8[rows, K], scales float[rows, K/128]:
 *                      s = amax / 448 (1 if amax = 0, 2^-149 if it rounds to 0),
 *                      q = e4m3 of clamp(y / s, -448, 448)
 *   (E4M3, MX)         codes uint8[rows, K], scales uint8[rows, K/32] (e8m0):
 *                      code = clamp(floor(log2 amax) - 8 + 127, 0, 254) (127 if amax = 0),
 *                      q = e4m3 of clamp(y 2^(127 - code), -448, 448)
 *   (E2M1, MX)         codes uint8[rows, K/2] (even K index in the low nibble), scales as above
 *                      with emax 2 in place of 8 and a clamp to +-6
 *   (E2M1, NV)         codes uint8[rows, K/2], scales uint8[rows, K/16] (e4m3):
 *                      s = e4m3 of min(amax / 6, 448) (1 if amax = 0, 2^-9 if it rounds to 0),
 *                      q = e2m1 of clamp(y / s, -6, 6)
 * amax is the block's largest |y|; divisions are fp32; elements round to nearest even and keep the
 * sign of y (a negative value that rounds to 0 gives -0). The layouts are bsgemm_grouped's A.
 * A block that holds a NaN or an infinity gets a scale that is not finite (E4M3 BLOCKWISE: amax / 448;
 * MX: 255, NaN; NV: 0x7f, NaN) with unspecified codes, so that a product's row with it is NaN. */
#define BSG_QUANT(elem, scale) ((uint32_t)(elem) | ((uint32_t)(scale) << 8))

#define BSG_ACT_NONE 0u
#define BSG_ACT_SWIGLU 1u   /* y = g / (1 + exp(-g)) * u, g and u the two halves of a row */

/*
 * bsgemm_quantize - rows, or the SwiGLU of rows, in a quantised form.
 *
 *   x       DEVICE [rows, K] (BSG_ACT_NONE) or [rows, 2 K] (BSG_ACT_SWIGLU: columns 0 .. K - 1 are g,
 *           K .. 2 K - 1 are u: the output of a gate_up product). 16-byte aligned.
 *   rows    >= 0 (0 is a no-op); rows * K at most 2^35; K > 0 a multiple of 128, at most 2^30
 *   q       DEVICE codes (output), 16-byte aligned;  scales DEVICE (output), float-aligned for BLOCKWISE
 * y is formed in fp32 and quantised without rounding to x's type first. SwiGLU: y is 0 for finite g < -87.3
 * (where |g / (1 + exp(-g))| is below 1.1e-36) and finite u; an infinite g of either sign gives a NaN.
 * Errors: BSG_ERR_FMT (x_dtype, act, q_fmt), BSG_ERR_SHAPE, BSG_ERR_NULL, BSG_ERR_ALIGN,
 * BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_quantize(const void* x, uint32_t x_dtype, uint32_t act, int32_t rows, int32_t K, uint32_t q_fmt,
                    void* q, void* scales, void* stream);

/*
 * bsgemm_swiglu_backward - gradient of y = g / (1 + exp(-g)) * u (a quantisation of y passes it through).
 *
 * With s = 1 / (1 + exp(-g)):   dg = dy u s (1 + g (1 - s)),   du = dy g s   (0 for g < -87)
 *
 *   dy  DEVICE [rows, K] in dtype;  x  DEVICE [rows, 2 K], g and u as for bsgemm_quantize; 16-byte aligned
 *   rows >= 0 (0 is a no-op); K > 0 a multiple of 8, at most 2^30; rows * K at most 2^34
 *   dx  DEVICE [rows, 2 K] in dtype (output): dg, then du. May be x (in place).
 * Errors: as bsgemm_quantize.
 */
int bsgemm_swiglu_backward(const void* dy, const void* x, uint32_t dtype, int32_t rows, int32_t K, void* dx,
                           void* stream);

/*
 * bsgemm_rms_norm_quantize - residual addition, RMS norm, and its output in a quantised form.
 *
 *   h = x + residual, rounded to dtype and stored in residual_out (residual NULL: h = x, not stored)
 *   rstd = 1 / sqrt(mean over the row of h^2 + eps)
 *   y = (h rstd) weight in fp32, quantised as q_fmt says
 *
 *   x, residual   DEVICE [rows, K] in dtype, 16-byte aligned; residual may be NULL
 *   weight        DEVICE [K] in dtype, 16-byte aligned
 *   rows 0 .. 2^22 - 1 (0 is a no-op), K a multiple of 128, at most 32768; eps >= 0 (> 0 if a row may be
 *   all zeros)
 *   residual_out  DEVICE [rows, K] in dtype (output); NULL exactly where residual is. May be
 *                 residual or x itself (in place).
 *   rstd          DEVICE float[rows] (output, for the gradient); may be NULL
 *   q, scales     DEVICE outputs, as for bsgemm_quantize
 * Errors: as bsgemm_quantize.
 */
int bsgemm_rms_norm_quantize(const void* x, const void* residual, const void* weight, uint32_t dtype, int32_t rows,
                             int32_t K, float eps, uint32_t q_fmt, void* residual_out, float* rstd, void* q,
                             void* scales, void* stream);

/*
 * bsgemm_rms_norm_backward - gradient of the norm above (the quantisation passes it through).
 *
 * With n = h rstd and g = dy weight:
 *   dx[r] = rstd (g - n mean(g n)) + dresidual[r]   (also the gradient of residual: h is their sum)
 *   dweight = sum over rows of dy n
 *
 *   dy, h, dresidual  DEVICE [rows, K] in dtype, 16-byte aligned; dresidual may be NULL (0)
 *   weight            DEVICE [K] in dtype;  rstd DEVICE float[rows], as stored by the forward
 *   dx                DEVICE [rows, K] in dtype (output);  dweight DEVICE float[K] (output)
 *   workspace         DEVICE, 16-byte aligned, at least bsgemm_rms_norm_backward_workspace_size bytes
 *                     (may be NULL if rows = 0, which sets dweight to 0)
 * Calls that share a workspace must be ordered. Errors: BSG_ERR_FMT, BSG_ERR_SHAPE (sizes, workspace too
 * small), BSG_ERR_NULL, BSG_ERR_ALIGN, BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_rms_norm_backward_workspace_size(int32_t rows, int32_t K, size_t* bytes);
int bsgemm_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                             const void* dresidual, uint32_t dtype, int32_t rows, int32_t K, void* dx,
                             float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * bsgemm_route_sort - top-k picks sorted by expert: counts, group layout, tile map and the row of
 * every pick, in one call.
 *
 *   counts[e]      as bsgemm_route_counts
 *   expert_offsets, tile_offsets, expert_ids   as bsgemm_build_tiles of counts (padded or packed)
 *   dest[i]        row of pick i: expert_offsets[e] + the number of earlier picks of its expert e, the
 *                  order of bsgemm_quantize_permute; -1 if its id is outside [0, num_experts) or the
 *                  row would be >= M
 *
 *   topk_ids       DEVICE int32[num_picks], usually [tokens, top_k] row-major
 *   num_picks 0 .. 2^24, num_experts 1 .. 4096, num_tiles >= 0, M >= 0
 *   counts int32[num_experts], expert_offsets int32[num_experts + 1], tile_offsets
 *   int32[num_tiles + 1], expert_ids int32[num_tiles], dest int32[num_picks]: DEVICE outputs
 *   workspace      DEVICE, 4-byte aligned, at least bsgemm_route_sort_workspace_size bytes; NULL where
 *                  that is 0 (up to 4096 picks, above 2048 experts 2048, which take a single launch)
 * Calls that share a workspace must be ordered.
 * Errors: BSG_ERR_SHAPE, BSG_ERR_NULL, BSG_ERR_ALIGN, BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_route_sort_workspace_size(int32_t num_picks, int32_t num_experts, size_t* bytes);
int bsgemm_route_sort(const int32_t* topk_ids, int32_t num_picks, int32_t num_experts, int32_t num_tiles,
                      int32_t padded, int32_t M, int32_t* counts, int32_t* expert_offsets,
                      int32_t* tile_offsets, int32_t* expert_ids, int32_t* dest, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * bsgemm_permute_rows - token rows to the rows of their picks.
 *
 *   out[dest[t, j]] = x[t]   for every pick with 0 <= dest[t, j] < M
 *   rows expert_offsets[e] + counts[e] .. expert_offsets[e + 1] - 1 (below M): zero bytes
 *   all other rows of out are untouched. Its gradient is bsgemm_combine_rows without weights.
 *
 *   x         DEVICE [tokens, row_bytes], any element type (rows, codes, or scales), 4-byte aligned
 *   row_bytes > 0, a multiple of 4 (16-byte accesses where row_bytes and both buffers are multiples
 *             of 16); tokens * ceil(row_bytes / 256) at most 2^25
 *   dest      DEVICE int32[tokens, top_k];  counts, expert_offsets: as bsgemm_route_sort wrote them
 *   out       DEVICE [M, row_bytes] (output)
 * Two picks with one dest (never so after bsgemm_route_sort) leave either row.
 * Errors: BSG_ERR_SHAPE, BSG_ERR_NULL, BSG_ERR_ALIGN, BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_permute_rows(const void* x, int32_t row_bytes, const int32_t* dest, int32_t tokens, int32_t top_k,
                        const int32_t* counts, const int32_t* expert_offsets, int32_t num_experts, int32_t M,
                        void* out, void* stream);

/*
 * bsgemm_combine_rows - the rows of a token's picks back to the token, weighted.
 *
 *   out[t] = sum over j (ascending, fp32) of weights[t, j] y[dest[t, j]]
 * A pick whose dest is outside [0, M) adds nothing and its row is not read; a token without any
 * pick left gets 0.
 *
 *   y        DEVICE [M, K] in dtype, 16-byte aligned;  out DEVICE [tokens, K] in dtype (output)
 *   dest     DEVICE int32[tokens, top_k]
 *   weights  DEVICE float[tokens, top_k], or NULL: all 1
 *   K > 0 a multiple of 8; tokens * ceil(K / 512) at most 2^25
 * Errors: BSG_ERR_FMT, BSG_ERR_SHAPE, BSG_ERR_NULL, BSG_ERR_ALIGN, BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_combine_rows(const void* y, uint32_t dtype, const int32_t* dest, const float* weights, int32_t tokens,
                        int32_t top_k, int32_t K, int32_t M, void* out, void* stream);

/*
 * bsgemm_combine_backward - gradient of the weighted bsgemm_combine_rows.
 *
 *   dy[dest[t, j]] = weights[t, j] dout[t];  dweights[t, j] = <dout[t], y[dest[t, j]]> (fp32), 0
 *   for a pick without a row. Padding rows of the groups (as in bsgemm_permute_rows) become zero in
 *   dy; all other rows of dy are untouched.
 *
 *   dout DEVICE [tokens, K], y and dy DEVICE [M, K] in dtype, 16-byte aligned; dweights DEVICE
 *   float[tokens, top_k] (output); dest, weights as above; counts, expert_offsets: the sort's
 *   tokens 0 .. 2^23, K > 0 a multiple of 8
 * Errors: as bsgemm_combine_rows.
 */
int bsgemm_combine_backward(const void* dout, const void* y, uint32_t dtype, const int32_t* dest,
                            const float* weights, int32_t tokens, int32_t top_k, int32_t K, const int32_t* counts,
                            const int32_t* expert_offsets, int32_t num_experts, int32_t M, void* dy,
                            float* dweights, void* stream);

/*
 * bsgemm_grouped_few_rows - the MX product of bsgemm_grouped for M-tiles of few rows (decode).
 *
 * Same operation, arguments and layouts as bsgemm_grouped with an MX fmt (without a schedule hint)
 * in which A or B (or both) is e2m1: e8m0 scales, any output type, packed or padded tile map or one
 * dense group. The weights are streamed once per tile and nothing is done for rows that are not there,
 * so it is the faster of the two while experts get few rows (bsgemm_grouped for more);
 * results agree up to the rounding order of fp32 sums. In pairs with an e4m3 operand the matrix instruction (here
 * and in bsgemm_grouped) cuts each product at 2^-13 of the largest among 8 consecutive K-elements.
 * Sizes: as bsgemm_grouped, K at most 2^22, tiles * N / 32 at most 2^21. M = 0 or no tiles: a no-op, in which A, B,
 * their scales and C may be NULL (so may expert_ids of no tiles).
 * Errors: BSG_ERR_FMT (also for the other scale kinds and e4m3 x e4m3), BSG_ERR_SHAPE, BSG_ERR_NULL,
 * BSG_ERR_ALIGN, BSG_ERR_DEVICE, BSG_ERR_LAUNCH.
 */
int bsgemm_grouped_few_rows(const void* A, const void* a_scales, const void* B, const void* b_scales,
                            const int32_t* expert_ids, const int32_t* tile_offsets, int32_t num_tiles, void* C,
                            int32_t M, int32_t N, int32_t K, int32_t num_experts, uint32_t fmt, void* stream);

/* Static, human-readable text for a bsg_status value (never NULL). */
const char* bsgemm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* BSGEMM_H */
