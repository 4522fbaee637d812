/*
 * moe_route.h -- C ABI of the GB300 (sm_103a) MoE routing + FP8 quantisation
 * hot path.
 *
 * Five operations, in the order a MoE layer runs them:
 *
 *   moe_topk_gate        scores [T,E] f32  -> topk_idx [T,k] i32, topk_weights [T,k] f32
 *   moe_route_map        topk_idx          -> counts [E], offsets [E+1], pos [T,k], sorted_src [T*k]
 *   moe_expand_cast_fp8  x [T,H] bf16, pos -> out [R,H] E4M3 bytes, out_sf [R,H/128] f32
 *   swiglu_cast_fp8      x [M,2N] bf16     -> out [M,N] E4M3 bytes, out_sf [M,N/128] f32
 *   moe_combine          y [R,H] bf16, topk_weights, pos -> out [T,H] bf16 or f32
 *
 * and their widened forms: the padded expert layout (moe_route_map_aligned,
 * moe_expand_cast_fp8_padded), the scale options and SwiGLU variants
 * (moe_expand_cast_fp8_ex, swiglu_cast_fp8_ex), the FP4 E2M1 casts
 * (moe_expand_cast_fp4, swiglu_cast_fp4), steps 1-3 in one call with a fused
 * decode launch (moe_route_expand_cast_fp8), and the route map without a
 * workspace (moe_route_map_noalloc); and the operators around the routed
 * experts (moe_block_norm, moe_balance_loss and moe_combine's gradient, with
 * their backward passes, and moe_expert_matvec_fp4), and a router with balance
 * and groups before 8-bit integer experts (moe_router_gate with its backward pass,
 * moe_cast_int8, moe_expert_matmul_int8).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers are DEVICE pointers into memory the caller owns (allocated by the
 *   caller, e.g. through PyTorch).  The library allocates no device memory and
 *   keeps no per-call state; a caller-provided workspace is the only scratch.
 * - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *   stream).  Every call only enqueues work on it and returns at once; no call
 *   synchronises except moe_get_device_status.
 * - Tensors are dense row-major with the shapes given; bf16 is passed as raw
 *   16-bit patterns, E4M3 (OCP E4M3FN: bias 7, max 448, no infinities) as raw
 *   bytes.
 * - Arguments are checked on the host BEFORE anything is launched.  A bad
 *   argument returns MOE_ERR_INVALID_ARG (or MOE_ERR_UNSUPPORTED for a valid
 *   but unimplemented option) and launches nothing.  A zero-sized problem
 *   returns MOE_OK and launches no kernel (moe_route_map with T == 0 still
 *   zero-fills counts and offsets with cudaMemsetAsync).
 * - Conditions only the data can reveal (an expert index outside [0,E), a
 *   pos row outside [0,num_rows)) are not memory errors: the kernel skips the
 *   offending access, and sets a bit in a device-side error word that
 *   moe_get_device_status reports and clears.
 * - A launch failure returns MOE_ERR_CUDA; moe_last_cuda_error_string gives
 *   the CUDA text.  No C++ exception crosses this boundary.
 * - Calls on distinct streams may run concurrently; the device error word is
 *   shared by all of them.
 * - Inputs must not contain NaN.  Results for NaN inputs are unspecified.
 *
 * Sources (page title, section):
 *   [TK]  "DeepSeek open-sources TileKernels: GPU operators written in Python
 *         approach hardware limits" (itsolotime.com): 2.1 Top-K Gating,
 *         2.2 Fused Expand, 3.1 quantisation config, 3.2 per-token cast,
 *         3.3 SwiGLU + quantisation, and the routing chain opening section 2.
 *   [PX]  "CuTeDSL at Perplexity" (perplexity.ai blog): MoE dispatch and
 *         combine, the TP=1 local kernel.
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ROUTE_ABI_VERSION 1

/* Largest supported expert count and top-k. */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 32
/* The FP8 casts' scaling group: one fp32 scale per 128 channels (the FP4
 * casts take 16, 32, 64 or 128). */
#define MOE_CAST_GROUP 128

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or range       */
    MOE_ERR_UNSUPPORTED = 2, /* valid request this library does not implement */
    MOE_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed          */
    MOE_ERR_DEVICE = 4       /* a kernel flagged bad data (see error bits)    */
} moe_status_t;

typedef enum moe_weight_mode {
    MOE_WEIGHTS_NONE = 0,        /* write topk_idx only                         */
    MOE_WEIGHTS_SOFTMAX_TOPK = 1 /* softmax over the k selected scores          */
} moe_weight_mode_t;

typedef enum moe_out_dtype {
    MOE_OUT_BF16 = 0,
    MOE_OUT_F32 = 1
} moe_out_dtype_t;

/* Scale options of the *_ex cast calls (bit flags). */
#define MOE_SF_COLMAJOR 0x1u /* scales transposed: [G][sf_ld] (TMA-aligned column-major) */
#define MOE_SF_POW2 0x2u     /* round_sf: smallest power of two >= the plain scale      */
#define MOE_SF_UE8M0 0x4u    /* store the power-of-two scale as its biased exponent
                                byte; requires MOE_SF_POW2.  Row-major: [rows][G] u8;
                                with MOE_SF_COLMAJOR: [ceil(G/4)][sf_ld] u32, four
                                consecutive groups of a row per word (group 4i+j in
                                byte j)                                                 */

/* Bits of the device error word (moe_get_device_status). */
#define MOE_DEVERR_EXPERT_RANGE 0x1u /* route_map: topk_idx outside [0, E)      */
#define MOE_DEVERR_POS_RANGE 0x2u    /* expand/combine: pos >= num_rows         */
#define MOE_DEVERR_DUPLICATE_EXPERT 0x4u /* route_map: a token names an expert twice */
#define MOE_DEVERR_ROWS_SHORT 0x8u   /* route_map_aligned: num_rows < padded total */
#define MOE_DEVERR_TIMEOUT 0x10u     /* a bounded wait inside a kernel ran out */
#define MOE_DEVERR_BOUNDS 0x20u      /* debug-bounds library only: an internal index
                                        or alignment check failed, access skipped */

/* Paths of moe_route_expand_cast_fp8. */
#define MOE_PATH_AUTO 0       /* the library's choice (see moe_route_expand_cast_fp8)     */
#define MOE_PATH_FUSED 1      /* one cooperative launch (decode shapes only)              */
#define MOE_PATH_SEPARATE 2   /* moe_topk_gate + moe_route_map + moe_expand_cast_fp8     */
#define MOE_PATH_REPLICATED 3 /* one ordinary launch, routing repeated per block (small T) */
#define MOE_PATH_CHAINED 4    /* three launches: top-k + chunk ranks, a scan, the expand   */
#define MOE_AUTO_REPLICATED_MAX_TOKENS 1024 /* AUTO's switch from REPLICATED to SEPARATE  */

/*
 * moe_topk_gate -- [TK] 2.1 Top-K Gating, plus the "Weight Normalization" that
 * closes [TK]'s routing chain, read as the softmax over the selected scores.
 *
 * For every token t the k experts with the largest scores[t, :], in
 * descending score order; equal scores go to the lower expert index (so the
 * result is unique).  -0.0 and +0.0 compare equal; +-inf are ordinary values.
 *   scores       [T, E] f32, read-only.
 *   topk_idx     [T, k] i32 out (the page's int64 narrowed: E <= 1024).
 *   topk_weights [T, k] f32 out, may be NULL when weight_mode is
 *                MOE_WEIGHTS_NONE; with MOE_WEIGHTS_SOFTMAX_TOPK,
 *                w[t,j] = exp(s_j - s_0) / sum_i exp(s_i - s_0) over the k
 *                selected scores s_0 >= s_1 >= ... (fp32, expf); scores must
 *                be finite.
 * Requires 1 <= E <= MOE_MAX_EXPERTS, 1 <= k <= min(E, MOE_MAX_TOPK), T >= 0,
 * scores 4-byte aligned.
 */
moe_status_t moe_topk_gate(const float *scores, int64_t num_tokens,
                           int32_t num_experts, int32_t num_topk,
                           int32_t *topk_idx, float *topk_weights,
                           int32_t weight_mode, void *stream);

/*
 * moe_route_map_workspace_bytes -- device scratch moe_route_map needs for a
 * problem of this size: a histogram row of E int32 per chunk of consecutive
 * tokens (chunks of a multiple of 32 tokens, at most 512, aiming at about 128
 * chunks), rounded up to 256 bytes.  0 when num_tokens == 0 or k is out of
 * range.  Pure host function.
 */
size_t moe_route_map_workspace_bytes(int64_t num_tokens, int32_t num_experts,
                                     int32_t num_topk);

/*
 * moe_route_map -- [PX] local dispatch: "count the tokens assigned to each
 * expert and give each token a unique index in its expert's list", made
 * stable and deterministic (the page's shared-memory atomics are not):
 *   counts[e]     = #{(t,j) : topk_idx[t,j] == e}                 [E]   i32
 *   offsets[e]    = sum_{e' < e} counts[e'], offsets[E] = T*k     [E+1] i32
 *   pos[t,j]      = offsets[e] + #{(t',j') before (t,j) in row-major
 *                   order with topk_idx[t',j'] == e}              [T,k] i32
 *   sorted_src[r] = t*k + j for r = pos[t,j]   (inverse of pos)   [T*k] i32
 * Rows of one expert are therefore in ascending token order.
 *   workspace: at least moe_route_map_workspace_bytes(...) bytes of device
 *   memory, 16-byte aligned; contents on entry are ignored; it is busy until
 *   the work enqueued on `stream` completes.  (For T <= 1024, E <= 256 and
 *   T*k <= 16384 the map is built in one launch in which every block builds
 *   it in shared memory and writes its own tokens' entries; the workspace is
 *   then not touched.  Otherwise a histogram launch and a rank launch.)
 * Each token's k experts must be distinct (as moe_topk_gate produces them); a
 * repeated expert sets MOE_DEVERR_DUPLICATE_EXPERT and leaves that token's
 * results unspecified (no write leaves the output buffers).  An index outside
 * [0, E) sets MOE_DEVERR_EXPERT_RANGE; that copy is not counted, its pos is
 * -1, and sorted_src keeps holes at its end.
 * Requires the same E and k limits as moe_topk_gate and T*k < 2^31.
 */
moe_status_t moe_route_map(const int32_t *topk_idx, int64_t num_tokens,
                           int32_t num_experts, int32_t num_topk,
                           int32_t *counts, int32_t *offsets, int32_t *pos,
                           int32_t *sorted_src, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * moe_route_map_aligned -- the route map into a padded expert layout, for an
 * expert GEMM that wants every expert's rows to start on a tile boundary
 * ([PX] dispatch: "tokens are optionally copied into padded buffers for the
 * MoE GEMM"; [TK] 2.2: rows no token lands on are zero-filled by the expand).
 * As moe_route_map, except that each expert's segment is rounded up to a
 * multiple of `align` rows:
 *   offsets[e+1]  = offsets[e] + align * ceil(counts[e] / align)
 *   pos[t,j]      = offsets[e] + rank of the copy among e's copies
 *   sorted_src[r] = t*k + j for r = pos[t,j]; -1 for every other row of
 *                   [0, num_rows) (padding rows and the tail)   [num_rows] i32
 * counts[e] is the unpadded count.  align == 1 gives moe_route_map's results
 * (with a -1 tail when num_rows > T*k).
 *   num_rows: rows of the padded buffers; T*k + E*(align-1) always suffices.
 *   If it is smaller than offsets[E] the kernel sets MOE_DEVERR_ROWS_SHORT and
 *   drops the copies that would land at or past num_rows (their pos is -1).
 * Requires 1 <= align <= 4096, T*k + E*(align-1) < 2^31 and num_rows < 2^31;
 * the workspace is moe_route_map_workspace_bytes(T, E, k).
 */
moe_status_t moe_route_map_aligned(const int32_t *topk_idx, int64_t num_tokens,
                                   int32_t num_experts, int32_t num_topk,
                                   int32_t align, int64_t num_rows, int32_t *counts,
                                   int32_t *offsets, int32_t *pos, int32_t *sorted_src,
                                   void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * moe_route_map_noalloc -- moe_route_map for callers that cannot allocate
 * device memory.  The pages have no counterpart: it exists for callers such
 * as engine plugins or runtimes that hand out every device buffer from their
 * own arena and forbid allocation while they run, so they cannot provide the
 * workspace moe_route_map needs.  Same arguments and results as
 * moe_route_map, minus the workspace; its histogram lives instead in one
 * static device array of MOE_ROUTE_NOALLOC_SCRATCH_BYTES that every GPU
 * loading this library holds until the process exits.
 * - Allocates nothing (no cudaMalloc, cudaFree or allocating library call).
 * - Returns MOE_ERR_UNSUPPORTED, launching nothing, when the problem needs
 *   more than that: moe_route_map_workspace_bytes(T, E, k) >
 *   MOE_ROUTE_NOALLOC_SCRATCH_BYTES.  Every problem with T <= 65536 fits
 *   (any E, k); larger ones fit while ceil(T / 512) * E <= 2^18.
 * - The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.
 * - All calls share the one array.  Nothing in it needs clearing (each call
 *   writes every entry it reads), but calls that overlap on the GPU (other
 *   streams, other threads) race on it and give wrong results: serialise them.
 * - Argument checks, including 4-byte alignment of every array, and data
 *   errors are those of moe_route_map: an expert index outside [0, E) or a
 *   token naming one expert twice sets its bit in the device error word that
 *   moe_get_device_status reports.
 */
#define MOE_ROUTE_NOALLOC_SCRATCH_BYTES (1u << 20)
moe_status_t moe_route_map_noalloc(const int32_t *topk_idx, int64_t num_tokens,
                                   int32_t num_experts, int32_t num_topk,
                                   int32_t *counts, int32_t *offsets,
                                   int32_t *pos, int32_t *sorted_src,
                                   void *stream);

/*
 * moe_expand_cast_fp8 -- [TK] 3.2 per_token_cast fused with [TK] 2.2
 * expand_to_fused.  For every token t and 128-channel group g of x[t, :]:
 *   amax   = max |x| over the group (bf16 widened exactly to f32)
 *   sf     = max(amax, 1e-4f) / 448   (f32, IEEE round-to-nearest-even;
 *            1e-4 is [TK] 3.1's E4M3 clamp_min_value)
 *   sf_inv = 1 / sf                   (f32, IEEE; "multiply by the inverse")
 *   q      = E4M3(x * sf_inv)         (f32 product, round to nearest even,
 *            saturating to +-448; the sign of zero is kept)
 * and for every j with pos[t,j] >= 0 the row of codes goes to
 * out[pos[t,j], :] and the group scales to out_sf[pos[t,j], :].  pos[t,j] < 0
 * means "no copy" ([TK] 2.2).  Rows of out no pos names are not written.
 *   x       [T, H] bf16, 16-byte aligned.      pos [T, k] i32.
 *   out     [num_rows, H] u8, 16-byte aligned. out_sf [num_rows, H/128] f32.
 * Requires H % 128 == 0, 1 <= k <= MOE_MAX_TOPK, num_rows < 2^31, group ==
 * 128 and T * H/128 < 2^31 (else MOE_ERR_UNSUPPORTED).  pos >= num_rows sets
 * MOE_DEVERR_POS_RANGE and is skipped.
 */
moe_status_t moe_expand_cast_fp8(const void *x, int64_t num_tokens,
                                 int32_t hidden, int32_t num_topk,
                                 const int32_t *pos, int64_t num_rows,
                                 uint8_t *out, float *out_sf, int32_t group,
                                 void *stream);

/*
 * moe_expand_cast_fp8_padded -- moe_expand_cast_fp8 into a padded layout,
 * zero-filling in the same launch every row r < num_rows with
 * sorted_src[r] < 0 ([TK] 2.2: the expand kernel's grid covers max(T, rows)
 * so that the invalid rows are zeroed without another launch).  Those rows get
 * all-zero codes and all-zero scales; rows named by pos are written as
 * moe_expand_cast_fp8 writes them.  sorted_src: [num_rows] i32 as
 * moe_route_map_aligned returns it.  Same requirements and error bits as
 * moe_expand_cast_fp8.
 */
moe_status_t moe_expand_cast_fp8_padded(const void *x, int64_t num_tokens,
                                        int32_t hidden, int32_t num_topk,
                                        const int32_t *pos, const int32_t *sorted_src,
                                        int64_t num_rows, uint8_t *out, float *out_sf,
                                        int32_t group, void *stream);

/*
 * moe_expand_cast_fp8_ex -- moe_expand_cast_fp8 with the scale options of
 * [TK] 3.1 (round_sf, packed UE8M0) and [TK] 2.2 (TMA-aligned column-major
 * scales), and optionally the zero-fill of moe_expand_cast_fp8_padded.
 *   sf_flags: 0 or a combination of MOE_SF_COLMAJOR, MOE_SF_POW2,
 *             MOE_SF_UE8M0 (which requires MOE_SF_POW2):
 *     0                      out_sf [num_rows][G] f32 (moe_expand_cast_fp8's)
 *     COLMAJOR               out_sf [G][sf_ld] f32
 *     POW2 (| COLMAJOR)      as above, scale = smallest power of two >=
 *                            max(amax, 1e-4)/448 (codes use its exact inverse)
 *     UE8M0|POW2             out_sf [num_rows][G] u8: biased exponent (value
 *                            2^(byte-127)) of the power-of-two scale
 *     UE8M0|POW2|COLMAJOR    out_sf [ceil(G/4)][sf_ld] u32, group 4i+j of row r
 *                            in byte j of word [i][r]
 *   sf_ld: column-major leading dimension, >= num_rows and a multiple of 4
 *          (16-byte aligned columns for TMA); ignored without COLMAJOR.
 *   sorted_src: NULL, or [num_rows] i32 to zero-fill the rows with a negative
 *          entry (codes 0, scales 0.0 or byte 0) in the same launch.
 *   workspace, workspace_bytes: NULL / 0, or device memory (16-byte aligned)
 *          of at least moe_expand_cast_fp8_ex_workspace_bytes(num_tokens,
 *          hidden, sf_flags) bytes.  With a column-major layout, sorted_src
 *          and a workspace, each token's scales are staged there once and a
 *          second kernel writes the column-major buffer row by row from
 *          sorted_src, in whole 128-byte lines; sorted_src must then be pos's
 *          inverse (as moe_route_map / moe_route_map_aligned return it), and
 *          a sorted_src entry >= num_tokens * num_topk sets
 *          MOE_DEVERR_POS_RANGE and gives that row zero scales.  Otherwise each copy's scales are
 *          stored directly (the same values; every store then writes part of
 *          an L2 sector, which at large num_rows is much slower).  Unused for
 *          row-major layouts.
 * Requirements and error bits as moe_expand_cast_fp8; out_sf 4-byte aligned
 * (1-byte for row-major UE8M0).
 */
moe_status_t moe_expand_cast_fp8_ex(const void *x, int64_t num_tokens, int32_t hidden,
                                    int32_t num_topk, const int32_t *pos,
                                    const int32_t *sorted_src, int64_t num_rows,
                                    uint8_t *out, void *out_sf, uint32_t sf_flags,
                                    int64_t sf_ld, void *workspace, size_t workspace_bytes,
                                    int32_t group, void *stream);

/* Workspace bytes moe_expand_cast_fp8_ex stages column-major scales in:
 * num_tokens * G * 4 (f32) or num_tokens * ceil(G/4) * 4 (packed UE8M0),
 * G = hidden / 128, rounded up to 256; 0 for row-major layouts. */
size_t moe_expand_cast_fp8_ex_workspace_bytes(int64_t num_tokens, int32_t hidden,
                                              uint32_t sf_flags);

/*
 * moe_expand_cast_fp4 -- expand + per-group FP4 E2M1 cast: [TK] 3.1
 * (CastOutputConfig with the float4_e2m1fn output type, clamp_min_value =
 * max_value * 2^-126 = 6 * 2^-126), 3.2 (per-group absmax -> scale ->
 * multiply by the scale's inverse, num_per_channels channels per group) and
 * 2.2 (copy to the rows pos names).
 *   scale of a group: fl32(max(amax, 6 * 2^-126) / 6), or the smallest power
 *   of two >= it under MOE_SF_POW2; code = E2M1(fl32(x * fl32(1 / scale))),
 *   round to nearest, ties to the even code, saturating at +-6, the sign kept
 *   (also for zero).  E2M1 (OCP MX FP4): sign bit 3, exponent bits 2..1 with
 *   bias 1, mantissa bit 0; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   out: [num_rows][H/2] u8, two codes per byte, element 2i in the low nibble.
 *   out_sf, sf_flags, sf_ld, sorted_src, workspace: as moe_expand_cast_fp8_ex,
 *   with G = H / group scales per row.
 *   group: 16, 32, 64 or 128 channels per scale.
 * Requires H % 32 == 0, H % group == 0, H <= 16384, 1 <= k <= MOE_MAX_TOPK,
 * num_rows < 2^31, x and out 16-byte aligned.  Error bits as
 * moe_expand_cast_fp8.
 */
moe_status_t moe_expand_cast_fp4(const void *x, int64_t num_tokens, int32_t hidden,
                                 int32_t num_topk, const int32_t *pos, const int32_t *sorted_src,
                                 int64_t num_rows, uint8_t *out, void *out_sf, uint32_t sf_flags,
                                 int64_t sf_ld, void *workspace, size_t workspace_bytes,
                                 int32_t group, void *stream);

/* Workspace bytes moe_expand_cast_fp4 stages column-major scales in: as
 * moe_expand_cast_fp8_ex_workspace_bytes with G = hidden / group. */
size_t moe_expand_cast_fp4_workspace_bytes(int64_t num_tokens, int32_t hidden, int32_t group,
                                           uint32_t sf_flags);

/*
 * swiglu_cast_fp8 -- [TK] 3.3, plain form (no clamp, no top-k weight).  For
 * each row r and channel c < N, in f32:
 *   g = x[r, c] (left half, the gate), u = x[r, N + c] (right half, up)
 *   v = g / (1 + exp(-g)) * u
 * then the per-128-channel cast of moe_expand_cast_fp8 on v.
 *   x [M, 2N] bf16, 16-byte aligned; out [M, N] u8, 16-byte aligned;
 *   out_sf [M, N/128] f32.
 * Requires N % 128 == 0, group == 128 and M * N/128 < 2^31 (else
 * MOE_ERR_UNSUPPORTED).  exp and the division use the GPU's exp2 and
 * reciprocal units (__expf, __fdividef), so v is within a few ulps of the
 * correctly rounded f32 value, and an E4M3 code can differ by one step from a
 * host evaluation when v / sf lies that close to a rounding midpoint.
 */
moe_status_t swiglu_cast_fp8(const void *x, int64_t num_rows, int32_t n,
                             uint8_t *out, float *out_sf, int32_t group,
                             void *stream);

/*
 * swiglu_cast_fp8_ex -- swiglu_cast_fp8 with the variants of [TK] 3.3 and the
 * scale options of moe_expand_cast_fp8_ex:
 *   has_clamp, clamp: if has_clamp, g = min(g, clamp) and u = min(max(u,
 *              -clamp), clamp) before the activation (clamp >= 0, finite);
 *   weights:   NULL, or [M] f32: v = g / (1 + exp(-g)) * u * weights[r] (the
 *              routed copy's top-k weight, in expert-sorted row order);
 *   clamp_count: NULL, or one u64 in device memory to which the number of
 *              inputs the clamp changed is ADDED (zero it to count one call);
 *   sf_flags, sf_ld: as moe_expand_cast_fp8_ex, over M rows.
 * Requirements as swiglu_cast_fp8.
 */
moe_status_t swiglu_cast_fp8_ex(const void *x, int64_t num_rows, int32_t n, uint8_t *out,
                                void *out_sf, uint32_t sf_flags, int64_t sf_ld,
                                int32_t has_clamp, float clamp, const float *weights,
                                uint64_t *clamp_count, int32_t group, void *stream);

/*
 * swiglu_cast_fp4 -- swiglu_cast_fp8_ex with the FP4 E2M1 output of
 * moe_expand_cast_fp4: the same SwiGLU values (clamp, weight, clamp count),
 * cast per group of `group` channels (16, 32, 64 or 128) with scale
 * max(amax, 6 * 2^-126) / 6 (or its power-of-two round-up), codes packed two
 * per byte, element 2i in the low nibble: out [M][N/2] u8; scales as
 * swiglu_cast_fp8_ex with G = N / group.
 * Requires N % group == 0, N % 32 == 0, x and out 16-byte aligned.
 */
moe_status_t swiglu_cast_fp4(const void *x, int64_t num_rows, int32_t n, uint8_t *out,
                             void *out_sf, uint32_t sf_flags, int64_t sf_ld, int32_t has_clamp,
                             float clamp, const float *weights, uint64_t *clamp_count,
                             int32_t group, void *stream);

/*
 * moe_combine -- [PX] combine: "accumulate in registers using the token
 * positions, then write the final tokens".  For every token t:
 *   out[t, c] = sum_{j=0..k-1, pos[t,j] >= 0} topk_weights[t,j] * y[pos[t,j], c]
 * accumulated in f32 in slot order j = 0..k-1 (fused multiply-add), then
 * rounded to nearest even bf16 (MOE_OUT_BF16) or kept f32 (MOE_OUT_F32).
 *   y   [num_rows, H] bf16, 16-byte aligned (the expert outputs in the
 *       expert-sorted layout moe_route_map produced)
 *   topk_weights [T, k] f32, pos [T, k] i32
 *   out [T, H] bf16 or f32, 16-byte aligned
 * Requires H % 8 == 0 and T * H/8 < 2^31 (else MOE_ERR_UNSUPPORTED).
 * pos >= num_rows sets MOE_DEVERR_POS_RANGE and that copy contributes nothing.
 */
moe_status_t moe_combine(const void *y, const float *topk_weights,
                         const int32_t *pos, int64_t num_tokens, int32_t hidden,
                         int32_t num_topk, int64_t num_rows, void *out,
                         int32_t out_dtype, void *stream);

/*
 * moe_route_expand_cast_fp8 -- steps 1-3 of the path in one call: top-k gate +
 * softmax weights, route map, expand + per-token E4M3 cast, with exactly the
 * results of moe_topk_gate (MOE_WEIGHTS_SOFTMAX_TOPK), moe_route_map and
 * moe_expand_cast_fp8 (num_rows = T*k).
 *
 * The FUSED path is the decode specialisation of "CuTeDSL at Perplexity"
 * (prefill/decode kernels; MoE dispatch): one cooperative launch of one block
 * per SM.  Every warp selects its tokens' experts and every block casts its
 * tokens into shared memory; block 0 then builds the route map once all
 * blocks have arrived on a counter, and signals the others, which write their
 * rows.  Each wait is bounded (1 s); one that runs out sets
 * MOE_DEVERR_TIMEOUT.  It applies to T <= 2048, 32 < E <= 256, k <= 32,
 * T*k <= 16384, H <= 16384 (shared-memory staging permitting).  The
 * REPLICATED path has no wait on another block and no cooperative launch:
 * every block builds the whole route map in its own shared memory, then casts
 * and writes its own tokens' rows (and their pos and sorted_src entries).  For
 * T <= 32 it is one launch in which every block also selects the experts of
 * all T tokens (block 0 writes idx, w, counts and offsets); above, the top-k
 * kernel runs first and a second launch does the rest.  It applies to
 * T <= 2048, T*k <= 16384, 32 < E <= 256, k <= 32, H <= 8192.  The SEPARATE
 * path is the launches of the individual calls (three or four: the route map
 * is one launch for T <= 1024).  The CHAINED path is three launches: the
 * top-k kernel, one CTA per chunk of 16 to 64 consecutive tokens, also counts
 * each chunk's copies per expert and ranks every copy among its expert's
 * copies in the chunk; a scan turns the counts into per-chunk bases, the
 * counts and the offsets; the expand kernel places every copy itself (expert
 * offset + chunk base + rank), writing pos and sorted_src, then stores the
 * rows.  It applies to
 * 32 < E <= 256, k <= 32, H <= 16384 with H/128 % 4 == 0 and 16-byte aligned
 * out and out_sf.
 *   scores [T,E] f32; x [T,H] bf16; topk_idx [T,k] i32; topk_weights [T,k]
 *   f32; counts [E], offsets [E+1], pos [T,k], sorted_src [T*k] i32;
 *   out [T*k,H] u8; out_sf [T*k,H/128] f32.
 *   workspace: at least moe_route_expand_cast_fp8_workspace_bytes(T,E,k)
 *   bytes, 16-byte aligned.  Its first 256 bytes hold the FUSED and CHAINED
 *   paths' control words (the fused launch's arrival counters; the chained
 *   scan's count of finished CTAs): ZERO them once before the first call
 *   (each call leaves them zero; after a MOE_DEVERR_TIMEOUT, zero them
 *   again).  One workspace must not be used by two calls in flight at once.
 *   mode: MOE_PATH_AUTO, MOE_PATH_FUSED, MOE_PATH_REPLICATED or
 *   MOE_PATH_CHAINED (MOE_ERR_UNSUPPORTED where they do not apply) or
 *   MOE_PATH_SEPARATE.  AUTO
 *   takes the path measured fastest on GB300 for the shape: REPLICATED for
 *   T <= MOE_AUTO_REPLICATED_MAX_TOKENS where it applies (E = 256, k = 8,
 *   H = 4096, one call: 8.8 against 14.0 us at T = 16, 12.9 against 14.0 at
 *   T = 256, 15.0 against 16.0 at T = 512, 17.0 against 18.0 at T = 768,
 *   20.1 against 20.1 at T = 1024 (14.2 against 14.6 back to back); at
 *   T = 2048 the separate launches are faster back to back), else SEPARATE
 *   (the separate launches, chained by programmatic dependent launch, were
 *   as fast as the FUSED launch for T <= 64 and faster above: its single
 *   routing block and the cooperative launch cost more than the gaps they
 *   remove; and 1-2 % faster than CHAINED at T = 1024 to 65536: the chained
 *   top-k kernel, the scan and the expand's placement step take longer than
 *   the route map's two launches they replace).
 * Requirements as the individual calls; group == 128.
 */
moe_status_t moe_route_expand_cast_fp8(const float *scores, int64_t num_tokens,
                                       int32_t num_experts, int32_t num_topk, const void *x,
                                       int32_t hidden, int32_t *topk_idx, float *topk_weights,
                                       int32_t *counts, int32_t *offsets, int32_t *pos,
                                       int32_t *sorted_src, uint8_t *out, float *out_sf,
                                       void *workspace, size_t workspace_bytes, int32_t mode,
                                       int32_t group, void *stream);

/* 256 + moe_route_map_workspace_bytes(T, E, k). */
size_t moe_route_expand_cast_fp8_workspace_bytes(int64_t num_tokens, int32_t num_experts,
                                                 int32_t num_topk);

/*
 * ------------------------------------------------------------------------
 * The operators around the routed experts: the block's norms with its gate and
 * residual scale, the router's balance loss with its gradient, the combine's
 * gradient, and the experts' products with 4-bit weights for decode batches; then
 * the router with a bias for balance and groups, and the experts in 8-bit integers.
 * They have no counterpart on the pages; the formulas are given in full here.
 * The conventions above hold, with one widening: where a float argument says
 * "-inf allowed", -inf is an ordinary value.
 * ------------------------------------------------------------------------
 */

/* Element types of the norms' tensors, and of the combine's gradient. */
typedef enum moe_dtype {
    MOE_DT_BF16 = 0,
    MOE_DT_F32 = 1
} moe_dtype_t;

/* Shape of the block's gate, and what is applied to it first. */
#define MOE_GATE_NONE 0     /* no gate: g = 1                                 */
#define MOE_GATE_CHANNEL 1  /* [H] f32: one value per channel                 */
#define MOE_GATE_TOKEN 2    /* [T] f32: one value per token                   */
#define MOE_GATE_ELEMENT 3  /* [T, H] in the block's type                     */
#define MOE_GATE_ACT_NONE 0
#define MOE_GATE_ACT_SIGMOID 1 /* g = 1 / (1 + exp(-gate))                    */

/* Largest hidden size of the norms. */
#define MOE_NORM_MAX_HIDDEN 16384

/*
 * moe_block_norm -- the norms before and after a block, in one pass:
 *   rstd_post[t] = 1 / sqrt(mean_c y[t,c]^2 + eps)
 *   z[t,c] = y[t,c] * rstd_post[t] * post_weight[c]     (post_weight NULL: z = y)
 *   h[t,c] = residual[t,c] + scale * g[t,c] * z[t,c]    (y NULL: h = residual)
 *   rstd_pre[t] = 1 / sqrt(mean_c h[t,c]^2 + eps)
 *   n[t,c] = h[t,c] * rstd_pre[t] * pre_weight[c]       (pre_weight NULL: no n)
 * h is rounded to the stream's type when stored, and n is computed from h
 * before that rounding; every sum and product is f32.  A row whose squares sum
 * beyond f32's range (elements near 2^64) has the inverse norm 0.
 *   residual, h      [T, H] in stream_dtype; h may be residual itself (in place)
 *   y, n             [T, H] in block_dtype; y may be NULL (h is then not written)
 *   gate             see MOE_GATE_*; NULL exactly when gate_kind is MOE_GATE_NONE
 *   post_weight, pre_weight  [H] f32, each may be NULL (post_weight needs y)
 *   rstd_post, rstd_pre      [T] f32 out, each may be NULL; kept for the backward
 * Requires T >= 0, 1 <= H <= MOE_NORM_MAX_HIDDEN, T * H < 2^40, eps > 0 and
 * finite, scale finite, y or pre_weight given, n non-NULL exactly when
 * pre_weight is, and every tensor aligned to its element.  Fastest with H % 8 == 0
 * and every [T, H] and [H] tensor 32-byte aligned; with 16-byte alignment alone
 * rows go element by element, but for forward calls of fewer than 2^19 elements
 * and for H > 8192.
 */
moe_status_t moe_block_norm(const void *residual, int32_t stream_dtype, const void *y,
                            int32_t block_dtype, int64_t num_tokens, int32_t hidden,
                            const float *post_weight, const void *gate, int32_t gate_kind,
                            int32_t gate_act, float scale, const float *pre_weight, float eps,
                            void *h, void *n, float *rstd_post, float *rstd_pre, void *stream);

/*
 * moe_block_norm_backward -- gradients of moe_block_norm for the gradients
 * grad_h of h and grad_n of n, from the saved h, y and inverse norms:
 *   u = grad_n * pre_weight
 *   d[t,c] = grad_h + rstd_pre * u - h * rstd_pre^3 * mean_c(u * h)
 *   grad_residual = d
 *   grad_pre_weight[c] = sum_t grad_n * h * rstd_pre
 *   grad_gate = scale * d * z * g'     (g' = 1, or g (1 - g) for the sigmoid),
 *               summed over the tokens (CHANNEL) or the channels (TOKEN)
 *   b = scale * g * d
 *   grad_post_weight[c] = sum_t b * y * rstd_post
 *   grad_y = rstd_post * b * post_weight
 *            - y * rstd_post^3 * mean_c(b * post_weight * y)   (no post_weight: b)
 *   grad_h [T, H] stream_dtype, may be NULL (zero); grad_n [T, H] block_dtype and
 *   h [T, H] stream_dtype, both needed with pre_weight; y, gate as above;
 *   rstd_post needed with post_weight, rstd_pre with pre_weight.
 *   grad_residual [T, H] stream_dtype (may be grad_h itself); grad_y [T, H]
 *   block_dtype, needed with y; grad_post_weight, grad_pre_weight [H] f32, needed
 *   with their weights; grad_gate in the gate's shape and type, needed with it.
 * Sums over tokens are f32 partial sums of fixed runs of tokens, added in a fixed order:
 * the same inputs give the same bits.  T == 0 zero-fills the [H] gradients.
 *   workspace: moe_block_norm_backward_workspace_bytes(T, H) bytes, 16-byte aligned.
 */
moe_status_t moe_block_norm_backward(
    const void *grad_h, const void *grad_n, const void *h, int32_t stream_dtype, const void *y,
    int32_t block_dtype, int64_t num_tokens, int32_t hidden, const float *post_weight,
    const void *gate, int32_t gate_kind, int32_t gate_act, float scale, const float *pre_weight,
    const float *rstd_post, const float *rstd_pre, void *grad_residual, void *grad_y,
    float *grad_post_weight, void *grad_gate, float *grad_pre_weight, void *workspace,
    size_t workspace_bytes, void *stream);

size_t moe_block_norm_backward_workspace_bytes(int64_t num_tokens, int32_t hidden);

/* The router's probabilities in the balance loss. */
#define MOE_SCORE_SOFTMAX 0 /* p = softmax(scores)                             */
#define MOE_SCORE_SIGMOID 1 /* p = sigmoid(scores) / sum of the row's sigmoids  */

/*
 * moe_balance_loss -- per-expert counts and the router's auxiliary losses over
 * packed sequences.  Sequence i holds the tokens seq_offsets[i] <= t <
 * seq_offsets[i+1].  A token counts if it lies in a sequence, token_mask (if
 * given) is nonzero there, and its row has a score above -inf and no NaN; n_i is
 * the number of such tokens of sequence i.  Scores of a token that does not count
 * may hold anything.  Over the tokens that count:
 *   counts[i,e] = #{(t,j) : topk_idx[t,j] == e}
 *   probs[i,e]  = (1/n_i) sum_t p[t,e]
 *   balance[i]  = sum_e (E counts[i,e] / (k n_i)) * probs[i,e]
 *   z[i]        = (1/n_i) sum_t (log sum_e exp(scores[t,e]))^2
 * and all of them are 0 where n_i = 0.
 *   scores [T, E] f32 (-inf allowed, +inf not); topk_idx [T, k] i32
 *   seq_offsets [S+1] i32, non-decreasing, within [0, T]; NULL for one sequence
 *   of all T tokens (num_seqs 1);  token_mask [T] u8, may be NULL
 *   balance, z [S] f32; counts [S, E] i32; probs [S, E] f32; tokens [S] i32 (n_i)
 *   workspace: moe_balance_loss_workspace_bytes(T, E, S) bytes, 16-byte aligned
 *   (0 for small problems: it may then be NULL)
 * An index outside [0, E) is not counted and sets MOE_DEVERR_EXPERT_RANGE.
 * The same inputs give the same bits.  Requires the E and k limits of
 * moe_topk_gate, 1 <= num_seqs <= 65535 and 0 <= T < 2^31.
 */
moe_status_t moe_balance_loss(const float *scores, const int32_t *topk_idx, int64_t num_tokens,
                              int32_t num_experts, int32_t num_topk, int32_t score_func,
                              const int32_t *seq_offsets, int32_t num_seqs,
                              const uint8_t *token_mask, float *balance, float *z,
                              int32_t *counts, float *probs, int32_t *tokens, void *workspace,
                              size_t workspace_bytes, void *stream);

size_t moe_balance_loss_workspace_bytes(int64_t num_tokens, int32_t num_experts,
                                        int32_t num_seqs);

/*
 * moe_balance_loss_backward -- the router's score gradient: of both losses, and
 * (where grad_topk_weights is given) of the softmax weights of the selected
 * scores that moe_topk_gate returns.  With f_e = E counts[i,e] / (k n_i), taken
 * as constant, and q = softmax(scores):
 *   a_e = grad_balance[i] f_e / n_i
 *   grad_scores[t,e] = p_e (a_e - sum_e' p_e' a_e') [* (1 - sigmoid(scores)) for
 *                      MOE_SCORE_SIGMOID]
 *                    + (2 grad_z[i] / n_i) lse_t q_e
 *                    + w_j (grad_w_j - sum_j' w_j' grad_w_j')   where e = topk_idx[t,j]
 * A token that does not count (see moe_balance_loss) gets a row of zeros.
 *   counts, tokens: as moe_balance_loss returned them
 *   grad_balance, grad_z [S] f32, each may be NULL (zero)
 *   topk_idx [T, k] i32 (a token's experts distinct), topk_weights and
 *   grad_topk_weights [T, k] f32: all three, or grad_topk_weights NULL
 *   grad_scores [T, E] f32 out
 */
moe_status_t moe_balance_loss_backward(const float *scores, int64_t num_tokens,
                                       int32_t num_experts, int32_t num_topk, int32_t score_func,
                                       const int32_t *seq_offsets, int32_t num_seqs,
                                       const uint8_t *token_mask, const int32_t *counts,
                                       const int32_t *tokens, const float *grad_balance,
                                       const float *grad_z, const int32_t *topk_idx,
                                       const float *topk_weights, const float *grad_topk_weights,
                                       float *grad_scores, void *stream);

/*
 * moe_combine_backward -- gradients of moe_combine:
 *   grad_y[pos[t,j], c] = bf16(topk_weights[t,j] * grad_out[t,c])   for pos[t,j] >= 0
 *   grad_topk_weights[t,j] = sum_c grad_out[t,c] * y[pos[t,j], c]   (f32; 0 for pos < 0)
 *   grad_out [T, H] in grad_dtype (MOE_DT_*), y and grad_y [num_rows, H] bf16, all
 *   16-byte aligned; topk_weights, grad_topk_weights [T, k] f32; pos [T, k] i32, each
 *   row named at most once
 *   sorted_src: NULL (rows no pos names are not written), or [num_rows] i32 as the
 *   route map returns it: rows with a negative entry are zero-filled
 * Requirements and error bits as moe_combine.
 */
moe_status_t moe_combine_backward(const void *grad_out, int32_t grad_dtype, const void *y,
                                  const float *topk_weights, const int32_t *pos,
                                  const int32_t *sorted_src, int64_t num_tokens, int32_t hidden,
                                  int32_t num_topk, int64_t num_rows, void *grad_y,
                                  float *grad_topk_weights, void *stream);

#define MOE_MATVEC_MAX_ROWS (1 << 18) /* most rows of moe_expert_matvec_fp4 */

/* Scale types of moe_expert_matvec_fp4's weights: the row-major layouts that
 * moe_expand_cast_fp4 writes. */
#define MOE_WSF_F32 0   /* [E][M][K/group] f32                                     */
#define MOE_WSF_UE8M0 1 /* [E][M][K/group] u8, value 2^(byte - 127)                */

/*
 * moe_expert_matvec_fp4 -- products of routed rows with their expert's 4-bit
 * weights, for decode batches (few rows per expert):
 *   o[r, m] = sum_c x[src(r), c] * E2M1(w[e(r), m, c]) * w_sf[e(r), m, c / group]
 *   out[r, n] = o[r, n]                                        (M = N), or
 *   out[r, n] = o[r, n] / (1 + exp(-o[r, n])) * o[r, N + n]    (swiglu: M = 2N)
 * for the rows offsets[e] <= r < offsets[e+1] of every expert e, in f32, rounded
 * once to out_dtype.  Rows at or past offsets[E] are not written.
 * x enters the products scaled by a power of two per 256 channels and rounded to
 * f16: a channel is exact unless it is below 2^-31 of the largest of its 256, and
 * then off by less than 2^-39 of that.
 *   x [num_x, K] bf16, finite, 16-byte aligned
 *   w [E, M, K/2] u8, two E2M1 codes per byte, element 2i in the low nibble (the
 *   layout moe_expand_cast_fp4 writes), 16-byte aligned; w_sf as MOE_WSF_*, below
 *   2^100, 4-byte aligned
 *   offsets [E+1] i32, non-decreasing, within [0, num_rows], as the route maps
 *   return it; NULL (E == 1 only): all num_rows rows
 *   sorted_src: NULL: src(r) = r (num_x >= num_rows); or [num_rows] i32 as the route
 *   maps return it: src(r) = sorted_src[r] / num_topk, and a negative entry gives
 *   a row of zeros
 *   out [num_rows, N] in out_dtype (MOE_OUT_*)
 * group is 16, 32, 64 or 128; K % 32 == 0, K % group == 0, K <= 16384, M * K < 2^32,
 * E * M < 2^31, num_rows <= MOE_MATVEC_MAX_ROWS.  offsets
 * beyond num_rows or a src outside [0, num_x) set MOE_DEVERR_POS_RANGE; such rows
 * are not written, or are zero.  Every wait for a copy is bounded (1 s); one that
 * runs out sets MOE_DEVERR_TIMEOUT.
 */
moe_status_t moe_expert_matvec_fp4(const void *x, int64_t num_x, const uint8_t *w,
                                   const void *w_sf, int32_t sf_type, int32_t group,
                                   const int32_t *offsets, const int32_t *sorted_src,
                                   int32_t num_experts, int32_t num_topk, int64_t num_rows,
                                   int32_t k_dim, int32_t n_dim, int32_t swiglu, void *out,
                                   int32_t out_dtype, void *stream);

/* What a group of experts is ranked by in moe_router_gate. */
#define MOE_GROUP_MAX 0  /* its largest s + bias                                  */
#define MOE_GROUP_TOP2 1 /* the sum of its two largest (of one, if it has one)    */
#define MOE_MAX_GROUPS 32

/*
 * moe_router_gate -- the router of a block with balanced and grouped experts:
 *   s[t,e] = softmax over e of scores[t,e]            (MOE_SCORE_SOFTMAX), or
 *            1 / (1 + exp(-scores[t,e]))              (MOE_SCORE_SIGMOID);
 *            0 where scores[t,e] is -inf
 *   c[t,e] = s[t,e] + bias[e]                         (bias NULL: s[t,e])
 * The num_groups groups of E / num_groups consecutive experts are ranked by
 * group_score over their experts with scores above -inf (a group without any
 * comes last); the topk_groups first stay.  Of their experts the k with the largest
 * c are selected, in descending order; experts with a score of -inf come last.
 * Equal values go to the lower group and the lower expert.  Values are compared as
 * real numbers: in f32, and in f64 where f32 cannot tell them apart (also where the two
 * largest of a group nearly cancel, by biases of both signs).
 *   topk_weights[t,j] = scale * s_j / sum_j' s_j'     (renormalize; 0 if the sum is 0)
 *                       scale * s_j                   (otherwise)
 * with s_j the score of the j-th selected expert: the bias decides the selection
 * only.  The ratio of sigmoids keeps its digits however small they are.
 *   scores [T,E] f32 (-inf allowed, +inf not); bias [E] f32, below 2^100 in magnitude,
 *   may be NULL;
 *   topk_idx [T,k] i32, topk_weights [T,k] f32
 * Requires the E and k limits of moe_topk_gate, 1 <= num_groups <= MOE_MAX_GROUPS,
 * E % num_groups == 0, 1 <= topk_groups <= num_groups, k <= E / num_groups *
 * topk_groups and a finite scale.
 */
moe_status_t moe_router_gate(const float *scores, int64_t num_tokens, int32_t num_experts,
                             int32_t num_topk, int32_t score_func, const float *bias,
                             int32_t num_groups, int32_t topk_groups, int32_t group_score,
                             int32_t renormalize, float scale, int32_t *topk_idx,
                             float *topk_weights, void *stream);

/*
 * moe_router_gate_backward -- the score gradient of moe_router_gate's weights, for
 * their gradient g = grad_topk_weights and e = topk_idx[t,j] (the selection and the
 * bias get none).  With w and s as above:
 *   renormalize: grad_scores[t,e] = w_j (g_j - sum_j' g_j' w_j' / scale) [* (1 - s_j)
 *                                   for MOE_SCORE_SIGMOID]
 *   otherwise:   grad_scores[t,e] = scale g_j s_j (1 - s_j)            (sigmoid)
 *                grad_scores[t,e'] = s_e' (scale g_j [e' = e] - scale sum_j' g_j' s_j')
 *                                    for every expert e'               (softmax)
 * and 0 elsewhere; with add, that is added to add's entry (moe_balance_loss_backward's
 * gradient, say).  An expert that a token names twice gets both gradients.
 *   scores [T,E] f32 as above; topk_idx [T,k] i32; grad_topk_weights [T,k] f32;
 *   add [T,E] f32, may be NULL
 *   grad_scores [T,E] f32 out; may be add itself (in place)
 * An index outside [0, E) is left out of every sum and sets MOE_DEVERR_EXPERT_RANGE.
 * Requires the E and k limits of moe_topk_gate and a finite scale.
 */
moe_status_t moe_router_gate_backward(const float *scores, int64_t num_tokens,
                                      int32_t num_experts, int32_t num_topk, int32_t score_func,
                                      int32_t renormalize, float scale, const int32_t *topk_idx,
                                      const float *grad_topk_weights, const float *add,
                                      float *grad_scores, void *stream);

/*
 * moe_cast_int8 -- rows to 8-bit integers with one scale per row, for
 * moe_expert_matmul_int8 (activations: a row per token; weights: a row per output):
 *   a = max(max_c |x[t,c]|, 2^-96)
 *   out_sf[t] = a / 127;  out[t,c] = rint(x[t,c] * (127 / a))
 * each step in f32, rounded to nearest (ties to even): values in [-127, 127].
 *   x [T,H] in dtype (MOE_DT_*), finite; out [T,H] i8; out_sf [T] f32
 * Requires 0 <= T < 2^31, 1 <= H <= 2^30, T * H < 2^40 and every tensor aligned to its
 * element.
 * Fastest with H % 8 == 0, x 16-byte and out 8-byte aligned.
 */
moe_status_t moe_cast_int8(const void *x, int32_t dtype, int64_t num_rows, int32_t hidden,
                           int8_t *out, float *out_sf, void *stream);

/*
 * moe_expert_matmul_int8 -- products of routed 8-bit rows with their expert's 8-bit
 * weights, with a scale per row of x and per output channel:
 *   o[r, m] = (sum_c x[src(r), c] * w[e(r), m, c]) * x_sf[src(r)] * w_sf[e(r), m]
 *   out[r, n] = o[r, n]                                        (M = N), or
 *   out[r, n] = o[r, n] / (1 + exp(-o[r, n])) * o[r, N + n]    (swiglu: M = 2N)
 * for the rows offsets[e] <= r < offsets[e+1] of every expert e, from one row per
 * expert to all rows, rounded once to out_dtype; the scales are multiplied in the order
 * given, each product in f32.  Rows at or past offsets[E] are not written.  The sum of
 * products is a sum of f32 in a fixed order; it is exact while no
 * partial sum passes 2^24 (always so for K <= 1024).
 *   x [num_x, K] i8, 16-byte aligned; x_sf [num_x] f32
 *   w [E, M, K] i8, 16-byte aligned; w_sf [E, M] f32
 *   offsets [E+1] i32, non-decreasing, within [0, num_rows], as the route maps
 *   return it; NULL (E == 1 only): all num_rows rows
 *   sorted_src: NULL: src(r) = r (num_x >= num_rows); or [num_rows] i32 as the route
 *   maps return it: src(r) = sorted_src[r] / num_topk, and a negative entry gives
 *   a row of zeros
 *   out [num_rows, N] in out_dtype (MOE_OUT_*)
 * Requires K % 16 == 0, 16 <= K <= 65536, num_rows < 2^31, E * M < 2^31 - 512 and the
 * limits of E and k.  offsets beyond num_rows or a src outside [0, num_x) set
 * MOE_DEVERR_POS_RANGE; such rows are not written, or are zero.  Every wait inside the
 * kernel is bounded (1 s); one that runs out sets MOE_DEVERR_TIMEOUT, and the kernel ends
 * once its copies and products in flight have (out is then unspecified).
 * The kernel's form goes by num_rows, as the host does not know the experts' rows: with far
 * more rows in the buffer than experts have (padding, a buffer for the worst case), a form
 * for longer runs is taken than theirs.
 */
moe_status_t moe_expert_matmul_int8(const int8_t *x, const float *x_sf, int64_t num_x,
                                    const int8_t *w, const float *w_sf, const int32_t *offsets,
                                    const int32_t *sorted_src, int32_t num_experts,
                                    int32_t num_topk, int64_t num_rows, int32_t k_dim,
                                    int32_t n_dim, int32_t swiglu, void *out, int32_t out_dtype,
                                    void *stream);

/* Test hooks of the fused path and of moe_expert_matmul_int8, process-wide, read at each
 * launch:
 *   MOE_DEBUG_WAIT_TIMEOUT_NS: the bound of every wait of theirs (default 1e9 ns), but for
 *   those for the work in flight of a kernel that gives up, which stay at 1e9 ns;
 *   MOE_DEBUG_SKIP_ROUTE_SIGNAL: nonzero = block 0 never signals "routed", so
 *   the copy blocks' waits run out (the failure path, without a fault);
 *   MOE_DEBUG_WEIGHT_STAGES: how many stages of 128 channels of weights each CTA of the 8-bit
 *   products asks for in all, so that the waits for the next one run out; -1 (default): all.
 * Returns MOE_ERR_INVALID_ARG for an unknown key or a value out of range. */
#define MOE_DEBUG_WAIT_TIMEOUT_NS 1
#define MOE_DEBUG_SKIP_ROUTE_SIGNAL 2
#define MOE_DEBUG_WEIGHT_STAGES 3
moe_status_t moe_debug_set(int32_t key, int64_t value);

/* Which form of its kernel moe_expert_matmul_int8 takes on the current device for a call
 * with these sizes and offsets given, for tests: a cluster of CTAs per tile, each with a
 * part of the channels (few tiles); a CTA per tile; or a pair of CTAs per tile (more than
 * 104 rows per expert, counting every row of out). */
#define MOE_MATMUL_INT8_CLUSTER 1
#define MOE_MATMUL_INT8_CTA 2
#define MOE_MATMUL_INT8_PAIR 3
moe_status_t moe_debug_matmul_int8_form(int32_t num_experts, int64_t num_rows, int32_t k_dim,
                                        int32_t n_dim, int32_t swiglu, int32_t *form);

/*
 * moe_debug_cvt -- the device's value conversions on arbitrary f32 input, for
 * tests: out[i] = the E4M3FN code (MOE_DEBUG_CVT_E4M3: round to nearest even,
 * saturating at +-448, NaN -> NaN) or the E2M1 code in the low nibble
 * (MOE_DEBUG_CVT_E2M1: round to nearest even, saturating at +-6) of in[i],
 * exactly as the cast kernels convert x * (1 / scale).
 *   in [n] f32, out [n] u8, both 16-byte aligned; n % 4 == 0.
 */
#define MOE_DEBUG_CVT_E4M3 0
#define MOE_DEBUG_CVT_E2M1 1
moe_status_t moe_debug_cvt(int32_t format, const float *in, uint8_t *out, int64_t n,
                           void *stream);

/*
 * moe_peak_copy -- a plain 16-byte vectorised device-to-device copy of
 * `bytes` bytes (a multiple of 16; both pointers 16-byte aligned), used to
 * measure the HBM bandwidth the kernels above are held against.
 */
moe_status_t moe_peak_copy(const void *src, void *dst, size_t bytes, void *stream);

/*
 * moe_get_device_status -- synchronises `stream`, then reads and clears the
 * current device's error word.  Returns MOE_OK when no bit was set,
 * MOE_ERR_DEVICE when one was (the bits go to *error_bits if non-NULL), or
 * MOE_ERR_CUDA if synchronising failed.
 */
moe_status_t moe_get_device_status(void *stream, uint32_t *error_bits);

/* Static description of a status code (never NULL). */
const char *moe_status_string(moe_status_t status);

/* Text of the last CUDA error seen by this library on the calling thread. */
const char *moe_last_cuda_error_string(void);

/* MOE_ROUTE_ABI_VERSION of the loaded library. */
int32_t moe_abi_version(void);

/* Number of kernels this library has launched in this process so far. */
uint64_t moe_kernel_launch_count(void);

/*
 * Debug-bounds build.  The same sources compiled with MOE_DEBUG_BOUNDS
 * defined give libmoe_route_debug.so (the Python binding loads it when the
 * environment variable MOE_DEBUG_BOUNDS is 1).  Its kernels check, before the
 * access each guards, invariants that the normal build takes from the kernels'
 * construction: the alignment, size and place in shared memory of every TMA
 * copy, the alignment of wide scale stores, the shared-memory extent of the
 * staging slots, and the sorted_src row of every copy the decode kernels
 * place.  A failed check skips that access and sets MOE_DEVERR_BOUNDS; no
 * kernel traps.  Results are otherwise identical to the normal build's.
 *
 * moe_debug_bounds_enabled: 1 in the debug-bounds library, 0 otherwise.
 * moe_debug_bounds_selftest: in the debug-bounds library, launches one
 *   kernel whose single check is false by construction (it guards no memory
 *   access), so that the next moe_get_device_status reports
 *   MOE_DEVERR_BOUNDS; returns MOE_OK, or MOE_ERR_CUDA if the launch failed.
 *   In the normal library: MOE_ERR_UNSUPPORTED, nothing launched.
 */
int32_t moe_debug_bounds_enabled(void);
moe_status_t moe_debug_bounds_selftest(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_H */
