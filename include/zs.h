/*
 * zs.h -- C ABI of one data-parallel rank's sharded ZeRO/FSDP update on
 * AMD Instinct MI355X (gfx950).
 *
 * The update of one rank, in the order the pages give it:
 *   1. pack     zs_flat_layout + zs_pack_shard: the rank's fp32 slice of a
 *               FlatParameter (all parameters of a unit laid end to end and
 *               padded at the tail to a multiple of N).
 *   2. reduce   zs_reduce_grads: the fp32 mean of N per-rank gradient
 *               contributions for that slice -- the arithmetic a
 *               reduce-scatter performs for this rank.
 *   3. AdamW    zs_adamw_step: the local AdamW update of the fp32 master, m
 *               and v slice, optionally writing the bf16 result straight
 *               into the rank's slot of the all-gather buffer.
 *   4. cast and copy-out
 *               zs_cast_for_gather: fp32 master -> bf16 slot of the gather
 *               buffer; zs_copy_out: a gathered flat buffer -> per-parameter
 *               tensors (the unshard copy-out).
 *   Fused       zs_sharded_step: steps 2-3 (and the cast) in one pass.
 * And around the update, for the parameters that no matrix product stands for:
 *   embedding   zs_embed_forward, zs_embed_backward
 *   layer norm  zs_layer_norm_forward, zs_layer_norm_backward
 *   RMS norm    zs_rms_norm_forward, zs_rms_norm_backward (with the residual's
 *               addition; outputs and kept inputs in 8 bits)
 * For what the passes between keep:
 *   activations zs_activation_pack, zs_activation_unpack (8 bits)
 * And for the head, which may be the embedding's table:
 *   loss        zs_linear_cross_entropy_forward, zs_linear_cross_entropy_backward
 *
 * Pages (title, address) cited below:
 *   [L5]  "Lesson 5: ZeRO and FSDP", hpc.payai.win/train/lesson05.html
 *   [ZvF] "ZeRO vs FSDP", muhenan.com/post/zero-vs-fsdp
 *   [FZ3] "03 - FSDP (ZeRO-3): per-layer all-gather and reshard",
 *         llm-infra-atlas.github.io/parallel/01_dp/03_fsdp/
 *   [LAF] "FSDP" (Latent Atlas), process-cxr.github.io/ai-library/training/
 *         distributed-training/fsdp
 *   [DPZ] "Data parallelism and ZeRO memory sharding", jefxiong.cn/index.php/
 *         archives/aigc-fundamentals-zero.html
 *
 * Conventions common to every entry point:
 *   - Ownership: the caller owns every buffer (device data, descriptor tables,
 *     workspace). The library allocates no memory and keeps no state between
 *     calls, so calls on different streams are independent.
 *   - Execution: device work is enqueued on `stream` (NULL = the legacy
 *     default stream) and is asynchronous; results are valid once the
 *     stream has completed. No call synchronises.
 *   - Errors: arguments are checked on the host before anything is enqueued;
 *     a failed check returns a negative ZS_ERR_* code and enqueues nothing.
 *     A HIP launch failure returns ZS_ERR_HIP. A HIP error already pending on
 *     the calling thread when a call that launches work begins (left by an
 *     earlier, unrelated HIP call) is also returned as ZS_ERR_HIP, before
 *     anything is enqueued, and is left pending for the caller to read and
 *     clear (hipGetLastError). zs_status_string() names every code.
 *   - Launch shapes: chosen per call from the sizes and world size. The
 *     environment variables ZS_ADAMW_V, ZS_ADAMW_LDS, ZS_RANK_CHUNK,
 *     ZS_FUSED_G, ZS_FUSED_LDS, ZS_FUSED_BS, ZS_ACCUM_SHAPE, ZS_REDUCE_G and
 *     ZS_GRID_CAP override them for measurement sweeps, and are read only when
 *     ZS_TUNING=1 is set, once per process, at the first call; they change
 *     speed, never results.
 *   - Sizes are element counts (int64_t); n == 0 is a valid no-op.
 *   - bf16 values are passed as uint16_t bit patterns (the top half of an
 *     IEEE fp32). fp32 -> bf16 is round-to-nearest-even; NaN stays a quiet
 *     NaN with its sign; overflow goes to infinity.
 *   - Alignment: any element-aligned pointer is accepted. Inputs and fp32
 *     state on 16-byte boundaries (8-byte for bf16 contributions) take the
 *     vector path, whatever the alignment of a bf16 output (its 4-element
 *     groups are stored as one 8-byte or two 4-byte writes, or, when the
 *     output is 2 or 6 bytes past an 8-byte boundary, as aligned 8-byte
 *     words that straddle neighbouring groups); others take an element-wise
 *     path with the same results.
 */
#ifndef ZS_H_
#define ZS_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t zs_status;

#define ZS_OK 0
#define ZS_ERR_NULL (-1)      /* a required pointer is NULL                       */
#define ZS_ERR_SIZE (-2)      /* negative or inconsistent element count           */
#define ZS_ERR_WORLD (-3)     /* world size outside [1, ZS_MAX_WORLD]             */
#define ZS_ERR_RANK (-4)      /* rank outside [0, world)                          */
#define ZS_ERR_DTYPE (-5)     /* dtype code is not ZS_F32 or ZS_BF16 (ids: ZS_I32, ZS_I64) */
#define ZS_ERR_HPARAM (-6)    /* hyper-parameter not finite / out of range, step<1 */
#define ZS_ERR_SHARD (-7)     /* shard_numel != ceil(total / world)               */
#define ZS_ERR_WORKSPACE (-8) /* workspace missing or smaller than required       */
#define ZS_ERR_LAYOUT (-9)    /* descriptor table does not tile [0, total)        */
#define ZS_ERR_ALIGN (-10)    /* pointer not aligned to its element size          */
#define ZS_ERR_OVERLAP (-11)  /* an output buffer overlaps an input it may not     */
#define ZS_ERR_HIP (-100)     /* a HIP runtime call or kernel launch failed       */

/* Element types of gradient contributions and parameters. */
#define ZS_F32 0
#define ZS_BF16 1

/* Type of activations kept in 8 bits (zs_activation_pack). */
#define ZS_E4M3 4

/* Types of token and position ids. */
#define ZS_I32 2
#define ZS_I64 3

/* Largest number of simulated ranks one reduce may combine. */
#define ZS_MAX_WORLD 256

/*
 * One parameter of a unit, as laid out in its FlatParameter ([L5] s7.1 point 1;
 * [ZvF] s3, difference 1; [LAF] s5.1). Tables of these live in DEVICE memory
 * when passed to zs_pack_shard / zs_copy_out, and in HOST memory when passed
 * to zs_check_layout.
 *   ptr          device address of the parameter's contiguous (C-order) storage
 *   flat_offset  element offset of the parameter inside the flat buffer
 *   numel        element count of the parameter
 * A valid table lists the parameters in flat order and tiles [0, total):
 * flat_offset[0] == 0 and flat_offset[i+1] == flat_offset[i] + numel[i].
 */
typedef struct zs_param_desc {
  void* ptr;
  int64_t flat_offset;
  int64_t numel;
} zs_param_desc;

/*
 * AdamW hyper-parameters ([LAF] s9.3 lists lr, beta1, beta2, epsilon,
 * weight_decay). Given in double; the kernels derive fp32 constants from
 * them on the host. `step` is the 1-based step count t used for bias
 * correction 1 - beta^t.
 */
typedef struct zs_adamw_hparams {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  int64_t step;
} zs_adamw_hparams;

/*
 * zs_flat_layout -- FlatParameter layout of a unit (host only, no device work).
 * [L5] s7.1 points 1 and 3; [LAF] s5.1; [DPZ] s4.2 (contiguous split).
 *   numels[nparams]      element count of each parameter, in registration order
 *   world                data-parallel world size N (>= 1)
 *   align                S is rounded up to a multiple of `align` elements
 *                        (>= 1). 1 gives the pages' layout, P = ceil(T / N) * N.
 *                        64 puts every rank's slice of a bf16 gather buffer,
 *                        and every row of a bf16 [N, S] receive buffer, on a
 *                        128-byte line: slices and rows off it cost the single
 *                        pass up to 3% (slices, at n = 1,003,782,656, N = 8)
 *                        and 10% (rows, at n = 117,187,500, N = 64). The extra
 *                        padding is at the tail; parameter offsets do not move.
 *   offsets_out[nparams] receives flat_offset of each parameter (exclusive
 *                        prefix sum of numels); may be NULL
 *   total_out            receives T = sum(numels)
 *   padded_out           receives P = S * N (tail padding only)
 *   shard_out            receives S = ceil(T / N) rounded up to a multiple of
 *                        align, the per-rank slice length
 * All pointers are host pointers. Output pointers other than offsets_out may
 * be NULL. Errors: ZS_ERR_NULL (numels NULL with nparams > 0), ZS_ERR_SIZE
 * (nparams < 0, align < 1, a negative numel, or T or P overflowing int64),
 * ZS_ERR_WORLD.
 */
zs_status zs_flat_layout(const int64_t* numels, int32_t nparams, int32_t world, int64_t align,
                         int64_t* offsets_out, int64_t* total_out, int64_t* padded_out,
                         int64_t* shard_out);

/*
 * zs_check_layout -- verify on the host that a descriptor table (HOST memory)
 * tiles [0, total) in order and that every non-empty parameter has a non-NULL
 * pointer aligned to its element size (`dtype`: ZS_F32 sources 4 bytes, ZS_BF16
 * sources and copy-out destinations 2 bytes). Returns ZS_OK or ZS_ERR_NULL /
 * ZS_ERR_SIZE / ZS_ERR_LAYOUT / ZS_ERR_ALIGN / ZS_ERR_DTYPE. The pack and
 * copy-out kernels rely on these properties of the device table without
 * re-checking it, so callers build the device copy from a table that passed.
 */
zs_status zs_check_layout(const zs_param_desc* host_desc, int32_t nparams, int64_t total,
                          int32_t dtype);

/*
 * zs_pack_shard -- the rank's fp32 master slice of the padded FlatParameter.
 * [L5] s7.1 points 1 and 3; [LAF] s5.1; [L5] s2 (fp32 master, m, v per rank).
 *   d_desc[nparams]  DEVICE table describing the unit (see zs_param_desc);
 *                    parameters hold `src_dtype` elements (ZS_F32 or ZS_BF16)
 *   total_numel      T of the unit (the table must tile [0, T))
 *   world, rank      N and r
 *   align, shard_numel
 *                    the layout's rounding and S: shard_numel must equal the S
 *                    that zs_flat_layout gives for (T, N, align), otherwise
 *                    ZS_ERR_SHARD
 *   master[S]        receives flat[r*S + k] for k < S, as fp32 (bf16 sources
 *                    are widened exactly); positions at or past T are +0.0
 *   exp_avg[S], exp_avg_sq[S]
 *                    optional (NULL = untouched); set to +0.0 (fresh Adam state)
 * Device pointers: d_desc, master, exp_avg, exp_avg_sq and the table's ptrs.
 * master must not overlap any parameter. Errors: ZS_ERR_NULL, ZS_ERR_SIZE,
 * ZS_ERR_WORLD, ZS_ERR_RANK, ZS_ERR_DTYPE, ZS_ERR_SHARD, ZS_ERR_HIP.
 */
zs_status zs_pack_shard(const zs_param_desc* d_desc, int32_t nparams, int64_t total_numel,
                        int32_t src_dtype, int32_t world, int32_t rank, int64_t align,
                        int64_t shard_numel, float* master, float* exp_avg, float* exp_avg_sq,
                        hipStream_t stream);

/*
 * zs_reduce_grads -- mean of N gradient contributions for this rank's slice.
 * [DPZ] s3.1 (equations for g_r and g: the mean over ranks equals the
 * full-batch gradient); [L5] s3 ZeRO-1/2 step 1 (reduce-scatter keeps only
 * this rank's 1/N); [L5] s7.5 (reduce_dtype = float32).
 *   rows[world]   HOST array of `world` DEVICE pointers; rows[q] points at
 *                 contribution q for this slice, n elements of `dtype`
 *                 (ZS_BF16 or ZS_F32); unused (may be NULL) when n == 0.
 *                 The pointers travel by value in the kernel arguments, so a
 *                 launch captured into a HIP graph keeps them: a replay reads
 *                 the same row buffers.
 *                 Rows that start on 128-byte boundaries stream fastest: the
 *                 N rows of one [N, n] receive buffer whose row pitch is not a
 *                 multiple of 64 bytes start off the cache-line grid, and each
 *                 wave load then touches one line more (10% slower for the
 *                 single pass at n = 117,187,500, N = 64); pad the pitch.
 *                 A pitch that is a multiple of 2 MiB (what separate large
 *                 allocations give) measured fastest, 1-5% ahead of pitches
 *                 off it by 256 B to 64 KiB.
 *   grad_out[n]   DEVICE fp32 output: g[k] = (c_0[k] + c_1[k] + ... ) / N,
 *                 summed in fp32 in ascending q starting from c_0[k], then
 *                 one IEEE division by N (bit-identical for any launch shape)
 *   sumsq_out     optional DEVICE double: receives sum_k g[k]^2 (this
 *                 shard's partial of a global gradient norm, [DPZ] s6),
 *                 accumulated in fp64 in a fixed order: the same bits on
 *                 every call with the same n, N and dtype on devices with
 *                 the same number of compute units (the launch's tiles, and
 *                 so the order of the partial sums, follow the CU count)
 *   workspace     DEVICE scratch of at least zs_workspace_bytes(n) bytes,
 *                 required only when sumsq_out != NULL
 * grad_out may not overlap any row; sumsq_out and workspace may not overlap
 * each other, grad_out or a row (ZS_ERR_OVERLAP). Errors: ZS_ERR_NULL,
 * ZS_ERR_SIZE, ZS_ERR_WORLD, ZS_ERR_DTYPE, ZS_ERR_WORKSPACE, ZS_ERR_ALIGN,
 * ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_reduce_grads(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                          float* grad_out, double* sumsq_out, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/*
 * zs_reduce_grads_noalloc -- zs_reduce_grads for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc): the same arguments, results and errors without the
 * workspace. The sum of squares' partials live in the library's own scratch,
 * a static device array of ZS_NOALLOC_MAX_N / 256 + 256 doubles (8 MiB + 2 KiB)
 * that every device the library runs on holds until the process ends. The
 * call allocates nothing; its first call on a device looks up that device's
 * copy once.
 *   n > ZS_NOALLOC_MAX_N with sumsq_out != NULL: ZS_ERR_WORKSPACE (the scratch
 *   is too small); without a sum of squares any n is accepted.
 * All calls on one device share its scratch: two calls with a sum of squares
 * that overlap in time on one device (on different streams, or from different
 * threads) race and may return a wrong sum of squares. Serialise them. Nothing
 * in the scratch needs clearing: every call overwrites what it reads.
 */
#define ZS_NOALLOC_MAX_N (INT64_C(1) << 28)
zs_status zs_reduce_grads_noalloc(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                                  float* grad_out, double* sumsq_out, hipStream_t stream);

/* Bytes of workspace zs_reduce_grads / zs_accumulate_grads need for a sum of
 * squares over n elements: one fp64 partial per 256-element tile (at most
 * 2^24 - 1 of them) plus 256 second-level partials; 0 for n < 0. The contents
 * need no initialisation and are overwritten by every call that takes a sum of
 * squares. */
size_t zs_workspace_bytes(int64_t n);

/*
 * zs_adamw_step -- AdamW on the rank's fp32 slice, in place.
 * [L5] s3 (ZeRO-1/2 step 2; ZeRO-3 item 4: local update of the 1/N fp32
 * state, no communication); [DPZ] s4.2 (bias-corrected first step, eps
 * outside the root); [LAF] s8.2 step 6. Weight decay is decoupled.
 * Per element, with t = hp->step:
 *   m' = b1 m + (1 - b1) g;   v' = b2 v + (1 - b2) g^2
 *   theta' = theta (1 - lr wd) - (lr / (1 - b1^t)) m' / (sqrt(v' / (1 - b2^t)) + eps)
 *   master[n], exp_avg[n], exp_avg_sq[n]   DEVICE fp32, updated in place
 *   grad[n]                                DEVICE fp32 (e.g. zs_reduce_grads' output)
 *   hp                                     HOST pointer
 *   grad_scale    optional DEVICE fp32 scalar (NULL = 1): g is multiplied by
 *                 *grad_scale before the update (e.g. a gradient-clipping
 *                 coefficient computed on the device from sums of squares)
 *   bf16_out[n]   optional DEVICE bf16 output (NULL = skip): bf16(theta'),
 *                 typically the rank's slot of the all-gather buffer
 * No two of master, exp_avg, exp_avg_sq, grad and bf16_out may share bytes, and
 * grad_scale may not overlap an output (ZS_ERR_OVERLAP). Arrays that start on
 * 128-byte boundaries stream fastest: a wave's 1 KiB access to an array that
 * starts elsewhere straddles a partial cache line at each end, and a
 * partial-line write costs HBM a read-modify-write (a shard split into chunks
 * should split on multiples of 32 elements).
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_HPARAM (non-finite values, lr, eps
 * or wd < 0, betas outside [0, 1), step < 1), ZS_ERR_ALIGN, ZS_ERR_OVERLAP,
 * ZS_ERR_HIP.
 */
zs_status zs_adamw_step(float* master, float* exp_avg, float* exp_avg_sq, const float* grad,
                        int64_t n, const zs_adamw_hparams* hp, const float* grad_scale,
                        uint16_t* bf16_out, hipStream_t stream);

/*
 * zs_cast_for_gather -- bf16 copy of the rank's updated fp32 slice into its
 * slot of the all-gather buffer ([L5] s3 ZeRO-1/2 step 2 and Fig. 5-4: write
 * back the BF16 parameter shard; the slot of rank r starts at r*S).
 *   master[n]       DEVICE fp32 input
 *   gather_slot[n]  DEVICE bf16 output (the caller passes gather + r*S)
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_ALIGN, ZS_ERR_HIP.
 */
zs_status zs_cast_for_gather(const float* master, int64_t n, uint16_t* gather_slot,
                             hipStream_t stream);

/*
 * zs_copy_out -- unshard copy-out: per-parameter tensors from a gathered flat
 * bf16 buffer ([L5] s7.1 point 1: contiguous slices of the gathered
 * FlatParameter become each submodule's parameter; [FZ3] s1 and s3: the
 * all-gather result is copied out before compute).
 *   gathered[gathered_numel]  DEVICE bf16 flat buffer (P elements; the tail
 *                             pad is ignored)
 *   d_desc[nparams]           DEVICE table of destinations (bf16 elements);
 *                             must tile [0, total_numel)
 *   total_numel               T of the unit; must be <= gathered_numel
 * param i receives gathered[flat_offset_i .. flat_offset_i + numel_i).
 * Destinations may not overlap `gathered` or each other. Errors: ZS_ERR_NULL,
 * ZS_ERR_SIZE, ZS_ERR_HIP.
 */
zs_status zs_copy_out(const uint16_t* gathered, int64_t gathered_numel, const zs_param_desc* d_desc,
                      int32_t nparams, int64_t total_numel, hipStream_t stream);

/*
 * zs_sharded_step -- reduce, AdamW and the bf16 cast in one pass over the
 * slice: the same arithmetic as zs_reduce_grads followed by zs_adamw_step
 * (bit-identical results), without writing or re-reading the fp32 gradient.
 *   rows, world, dtype, n      as zs_reduce_grads
 *   master, exp_avg, exp_avg_sq, hp, bf16_out
 *                              as zs_adamw_step (bf16_out may be NULL)
 *   grad_scale    optional DEVICE fp32 scalar (NULL = 1): the mean gradient is
 *                 multiplied by *grad_scale before the update (a clipping
 *                 coefficient computed from a prior sum of squares)
 * Errors: union of the two calls' errors.
 */
zs_status zs_sharded_step(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                          float* master, float* exp_avg, float* exp_avg_sq,
                          const zs_adamw_hparams* hp, const float* grad_scale,
                          uint16_t* bf16_out, hipStream_t stream);

/*
 * zs_accumulate_grads -- sharded (ZeRO-2) gradient accumulation over micro-
 * batches: reduce this micro-batch's N contributions and add the mean into the
 * rank's fp32 accumulator ([L5] s3: ZeRO-2 reduce-scatters every micro-batch
 * and keeps only its 1/N; [L5] s2: the fp32 buffer costs 4P/N).
 *   rows, world, dtype, n     as zs_reduce_grads
 *   acc[n]        DEVICE fp32 accumulator:
 *                   first != 0:  acc = scale * mean
 *                   first == 0:  acc = acc + scale * mean
 *                 mean as in zs_reduce_grads (bit-identical); the product with
 *                 scale is skipped when scale == 1 (e.g. scale = 1/K for a
 *                 mean over K micro-batches)
 *   sumsq_out, workspace, workspace_bytes
 *                 optional: sum of squares of the updated acc (fp64), as in
 *                 zs_reduce_grads -- on the last micro-batch this is the
 *                 shard's partial of the global gradient norm
 * Errors: those of zs_reduce_grads, ZS_ERR_HPARAM (scale not finite).
 */
zs_status zs_accumulate_grads(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                              float* acc, float scale, int32_t first, double* sumsq_out,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * zs_accumulate_local -- unsharded (ZeRO-1) accumulation of one micro-batch's
 * local gradient in fp32 ([L5] s3: ZeRO-1 sums the full local gradient and
 * reduce-scatters once after the last micro-batch; [L5] s2: 4P per rank).
 *   grad[n]   DEVICE gradient of `dtype` (ZS_BF16 or ZS_F32)
 *   acc[n]    DEVICE fp32: first != 0: acc = grad (widened exactly);
 *             first == 0: acc = acc + grad
 * The accumulators of all ranks then go through zs_accumulate_grads (first=1,
 * scale=1/K) or zs_reduce_grads as fp32 contributions.
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_DTYPE, ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_accumulate_local(const void* grad, int32_t dtype, int64_t n, float* acc,
                              int32_t first, hipStream_t stream);

/*
 * zs_clip_coefficient -- global-norm clipping factor from per-shard sums of
 * squares ([DPZ] s6: the global norm needs every shard's partial; the combine
 * across ranks is an all-reduce in a multi-GPU job).
 *   partials[count]  DEVICE fp64 sums of squares (e.g. each rank's sumsq_out),
 *                    added in index order
 *   max_norm         the clipping threshold (finite, > 0)
 *   coef_out         DEVICE fp32: min(1, max_norm / (sqrt(total) + 1e-6)),
 *                    NaN if the total is NaN; pass it as grad_scale to
 *                    zs_adamw_step
 *   norm_out         optional DEVICE fp64: sqrt(total)
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE (count < 1), ZS_ERR_HPARAM, ZS_ERR_ALIGN, ZS_ERR_HIP.
 */
zs_status zs_clip_coefficient(const double* partials, int32_t count, double max_norm,
                              float* coef_out, double* norm_out, hipStream_t stream);

/*
 * Per-parameter dim-0 sharding (FSDP2 Shard(0); [L5] s7.2 and Fig. 5-5: each
 * parameter keeps its shape and is split on dim 0, a rank holding [H/N, D];
 * [FZ3] s4: DTensor sharded on dim 0, batched all-gather). A parameter with d0
 * rows of `rowsize` elements gives each rank c = ceil(d0/N) rows, rank r
 * holding rows [r*c, min((r+1)*c, d0)) zero-padded to c rows. A rank's shard
 * of a unit (also the all-gather input) is its padded chunks concatenated in
 * registration order, L elements; the all-gather output is the N shards one
 * after the other (N * L elements).
 *
 *   ptr           device address of the full parameter (C order)
 *   flat_offset   offset of the parameter in the unsharded unit (prefix sum of numels)
 *   numel         elements of the parameter (d0 * rowsize)
 *   chunk         elements per rank: ceil(d0 / N) * rowsize
 *   local_offset  offset of the parameter's chunk inside a rank's shard
 */
typedef struct zs_dim0_desc {
  void* ptr;
  int64_t flat_offset;
  int64_t numel;
  int64_t chunk;
  int64_t local_offset;
} zs_dim0_desc;

/*
 * zs_dim0_layout -- per-parameter chunk sizes and the rank-shard layout (host only).
 *   dim0[nparams], rowsize[nparams]  HOST arrays (a 0-d parameter: dim0 = rowsize = 1)
 *   chunk_out[nparams]               receives ceil(dim0/N) * rowsize (may be NULL)
 *   local_offsets_out[nparams]       receives the chunk offsets in a rank's shard (may be NULL)
 *   local_total_out                  receives L (may be NULL)
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE (negative or overflowing sizes), ZS_ERR_WORLD.
 */
zs_status zs_dim0_layout(const int64_t* dim0, const int64_t* rowsize, int32_t nparams, int32_t world,
                         int64_t* chunk_out, int64_t* local_offsets_out, int64_t* local_total_out);

/*
 * zs_check_dim0_layout -- verify a HOST table: flat offsets tile [0, total),
 * local offsets tile [0, local_total) with the chunk sizes, numel <= world *
 * chunk, and non-empty parameters have storage aligned to the element size of
 * `dtype` (as zs_check_layout). Returns ZS_OK or ZS_ERR_NULL / ZS_ERR_SIZE /
 * ZS_ERR_WORLD / ZS_ERR_LAYOUT / ZS_ERR_ALIGN / ZS_ERR_DTYPE.
 */
zs_status zs_check_dim0_layout(const zs_dim0_desc* host_desc, int32_t nparams, int32_t world,
                               int64_t total, int64_t local_total, int32_t dtype);

/*
 * zs_pack_shard_dim0 -- rank r's fp32 master shard under dim-0 sharding
 * (padding rows +0.0), with optional zeroed Adam moments.
 *   d_desc[nparams]  DEVICE table (see zs_dim0_desc); parameters hold src_dtype
 *   local_total      L; master, exp_avg, exp_avg_sq hold L fp32 elements (DEVICE)
 * The AdamW, cast and fused-step entry points apply to the shard unchanged.
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_WORLD, ZS_ERR_RANK, ZS_ERR_DTYPE,
 * ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_pack_shard_dim0(const zs_dim0_desc* d_desc, int32_t nparams, int32_t src_dtype,
                             int32_t world, int32_t rank, int64_t local_total, float* master,
                             float* exp_avg, float* exp_avg_sq, hipStream_t stream);

/*
 * zs_copy_out_dim0 -- unshard under dim-0 sharding: every parameter's rows
 * from the N ranks' regions of the gathered bf16 buffer (padding rows
 * dropped). A real scatter: parameter i's rows [r*c, ...) come from
 * gathered[r*L + local_offset_i ...].
 *   gathered[gathered_numel]  DEVICE bf16, gathered_numel >= world * local_total
 *   d_desc[nparams]           DEVICE table of bf16 destinations
 *   total                     T of the unit (sum of numels)
 * Errors: ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_WORLD, ZS_ERR_ALIGN, ZS_ERR_HIP.
 */
zs_status zs_copy_out_dim0(const uint16_t* gathered, int64_t gathered_numel,
                           const zs_dim0_desc* d_desc, int32_t nparams, int32_t world,
                           int64_t total, int64_t local_total, hipStream_t stream);

/*
 * Producers of parameter gradients. The entry points above take a parameter's
 * gradient as it is; the ones below compute it for the parameters of a unit
 * that no matrix product stands for -- embedding tables and the weights and
 * biases of layer norms -- next to the forward pass that reads them. Like
 * zs_accumulate_local they write a gradient where the update takes it from:
 *   first != 0:  grad = the sum (a fresh contribution, every element written)
 *   first == 0:  grad = grad + the sum (the accumulator of earlier
 *                micro-batches; with a bf16 grad each call rounds once more)
 * Rows are `dim` consecutive elements; `*_ld` is the distance between the
 * starts of two rows in elements (>= dim), and what lies between two rows is
 * neither read nor written. Any element-aligned pointer and any dim are
 * accepted; rows on 16-byte boundaries are fastest. Arithmetic is fp32, each
 * result rounded once to its type. The sums over rows run in an order that
 * depends on the sizes (and on the tokens) alone: the same call gives the same
 * bits. Sizes: n, rows and vocab below 2^31, dim below 2^24 (else ZS_ERR_SIZE).
 * Overlap checks take rows with the gaps between them: two arguments may not
 * interleave in one buffer. The stream's device must be the current one.
 */

/*
 * zs_embed_forward -- rows of an embedding table, scaled, optionally plus rows
 * of a position table.
 *   table[vocab, dim]     DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride table_ld
 *   pos_table[pos_rows, dim]
 *                         optional DEVICE (NULL = none), `dtype`, row stride pos_ld
 *   tokens[n], positions[n]
 *                         DEVICE ids, `index_type` ZS_I32 or ZS_I64; positions
 *                         is read only with a pos_table
 *   out[n, dim]           DEVICE, `out_dtype`, row stride out_ld:
 *                         out[i] = scale * table[tokens[i]] (+ pos_table[positions[i]])
 * An id outside of its table (below 0, or vocab / pos_rows and above: -100 or
 * the like for ignored places) selects a row of zeros; nothing outside the
 * tables is read. scale must be finite.
 * out may not overlap the tables or the ids. Errors: ZS_ERR_NULL, ZS_ERR_SIZE
 * (negative or too large sizes, a row stride below dim), ZS_ERR_DTYPE,
 * ZS_ERR_HPARAM, ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_embed_forward(const void* table, int32_t dtype, int64_t vocab, int64_t dim,
                           int64_t table_ld, const void* pos_table, int64_t pos_rows, int64_t pos_ld,
                           const void* tokens, const void* positions, int32_t index_type, int64_t n,
                           float scale, void* out, int32_t out_dtype, int64_t out_ld,
                           hipStream_t stream);

/* Bytes of workspace zs_embed_backward needs for n tokens of a [vocab, dim]
 * table (0 for sizes it refuses). The contents need no initialisation. */
size_t zs_embed_workspace_bytes(int64_t n, int64_t vocab, int64_t dim);

/*
 * zs_embed_backward -- gradient of an embedding table.
 *   dout[n, dim]       DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride dout_ld
 *   tokens[n]          DEVICE ids, `index_type` ZS_I32 or ZS_I64; ids outside of
 *                      [0, vocab) and the id `padding_idx` (any id outside of
 *                      the table, such as -1, for none) contribute nothing
 *   grad[vocab, dim]   DEVICE, `grad_dtype`, row stride grad_ld:
 *                      grad[v] = (first ? 0 : grad[v]) + scale * sum of dout[i]
 *                      over the i with tokens[i] == v. With first != 0 every
 *                      row is written (zeros where no token selects it), with
 *                      first == 0 only the rows that tokens select.
 *   workspace          DEVICE scratch of at least zs_embed_workspace_bytes(n,
 *                      vocab, dim) bytes on a 16-byte boundary; calls that may
 *                      run at the same time, and captured graphs that may be
 *                      replayed at the same time, need one each
 * For a position table, pass the positions as tokens. scale must be finite.
 * A token's rows are added in fp32 in the order of their positions, in pieces
 * of equal length, and the pieces in order.
 * No two of grad, dout, tokens and workspace may share bytes. Errors:
 * ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_DTYPE, ZS_ERR_HPARAM, ZS_ERR_WORKSPACE,
 * ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_embed_backward(const void* dout, int32_t dtype, int64_t dout_ld, const void* tokens,
                            int32_t index_type, int64_t n, int64_t vocab, int64_t dim,
                            int64_t padding_idx, float scale, void* grad, int32_t grad_dtype,
                            int64_t grad_ld, int32_t first, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

/*
 * zs_layer_norm_forward -- layer norm over the last dimension.
 *   x[rows, dim]       DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride x_ld
 *   weight[dim], bias[dim]
 *                      DEVICE, `wdtype` (ZS_F32 or ZS_BF16); either may be NULL
 *                      (ones, zeros)
 *   eps                finite in fp32, >= 0
 *   y[rows, dim]       DEVICE, `dtype`, row stride y_ld:
 *                      y = (x - mean) * rstd * weight + bias with
 *                      mean = sum(x) / dim, rstd = 1 / sqrt(sum((x - mean)^2) / dim + eps)
 *   mean[rows], rstd[rows]
 *                      optional DEVICE fp32 outputs (NULL = skip; the backward
 *                      pass needs both)
 * y may not overlap x, weight or bias, nor mean and rstd anything. Errors:
 * ZS_ERR_NULL, ZS_ERR_SIZE (dim < 1 with rows > 0 among them), ZS_ERR_DTYPE,
 * ZS_ERR_HPARAM, ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_layer_norm_forward(const void* x, int32_t dtype, int64_t x_ld, const void* weight,
                                const void* bias, int32_t wdtype, int64_t rows, int64_t dim,
                                double eps, void* y, int64_t y_ld, float* mean, float* rstd,
                                hipStream_t stream);

/* Bytes of workspace zs_layer_norm_backward needs for the weight's and bias's
 * gradient (0 for sizes it refuses). The contents need no initialisation. */
size_t zs_layer_norm_workspace_bytes(int64_t rows, int64_t dim);

/*
 * zs_layer_norm_backward -- gradients of layer norm.
 *   dy[rows, dim], x[rows, dim]
 *                      DEVICE, `dtype`, row strides dy_ld, x_ld
 *   weight[dim]        DEVICE, `wdtype`, or NULL (ones)
 *   mean[rows], rstd[rows]
 *                      DEVICE fp32, as zs_layer_norm_forward gives them
 *   dx[rows, dim]      DEVICE, `dtype`, row stride dx_ld: with xh = (x - mean) * rstd,
 *                      dx = rstd * (dy * weight - mean(dy * weight) - xh * mean(dy * weight * xh))
 *   dweight[dim], dbias[dim]
 *                      DEVICE, `grad_dtype`; either may be NULL (skipped):
 *                      dweight = (first ? 0 : dweight) + sum over rows of dy * xh,
 *                      dbias = (first ? 0 : dbias) + sum over rows of dy
 *   workspace          DEVICE scratch of at least zs_layer_norm_workspace_bytes(rows,
 *                      dim) bytes on a 16-byte boundary, required unless dweight and
 *                      dbias are both NULL or there are no rows; calls and graph replays that may run at
 *                      the same time need one each
 * rows == 0 with first != 0 sets dweight and dbias to zero. No output may
 * share bytes with an input, the workspace or another output. Errors:
 * ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_DTYPE, ZS_ERR_WORKSPACE, ZS_ERR_ALIGN,
 * ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                                 int32_t dtype, const void* weight, int32_t wdtype, const float* mean,
                                 const float* rstd, int64_t rows, int64_t dim, void* dx, int64_t dx_ld,
                                 void* dweight, void* dbias, int32_t grad_dtype, int32_t first,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Activations in 8 bits: codes[rows, dim] are e4m3 (sign, 4 bits of exponent, 3 of
 * mantissa, largest finite value 448, no infinity), scales[rows, ceil(dim / 128)]
 * fp32, one for each block of 128 consecutive elements of a row (the last may be
 * short); a value is code * scale. A block's scale is the smallest power of two,
 * at least 2^-117, with which its largest finite magnitude stays within 448 (1
 * where all are zero): values are rounded once, to nearest even, and what they
 * stand for is exact in bf16 and fp32. Infinities and NaN become NaN, and are no
 * measure of the scale; magnitudes above 1.875 * 2^127 become that.
 */

/*
 * zs_activation_pack -- rows in 8 bits.
 *   x[rows, dim]       DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride x_ld
 *   codes[rows, dim]   DEVICE, row stride codes_ld
 *   scales[rows, ceil(dim / 128)]
 *                      DEVICE fp32, row stride scales_ld
 * No output may share bytes with another argument. Errors: ZS_ERR_NULL,
 * ZS_ERR_SIZE, ZS_ERR_DTYPE, ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_activation_pack(const void* x, int32_t dtype, int64_t x_ld, int64_t rows, int64_t dim,
                             uint8_t* codes, int64_t codes_ld, float* scales, int64_t scales_ld,
                             hipStream_t stream);

/*
 * zs_activation_unpack -- out[rows, dim] = code * scale, in `dtype` (ZS_F32 or
 * ZS_BF16) with row stride out_ld. Other scales than those of the calls here are
 * taken as they are, and products rounded. Otherwise as above.
 */
zs_status zs_activation_unpack(const uint8_t* codes, int64_t codes_ld, const float* scales,
                               int64_t scales_ld, int64_t rows, int64_t dim, void* out, int32_t dtype,
                               int64_t out_ld, hipStream_t stream);

/*
 * zs_rms_norm_forward -- root-mean-square norm over the last dimension, with the
 * residual's addition before it and an output in 8 bits.
 *   x[rows, dim]       DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride x_ld
 *   residual[rows, dim]
 *                      optional DEVICE (NULL = none), `sum_dtype`, row stride residual_ld
 *   sum[rows, dim]     optional DEVICE output, `sum_dtype`, row stride sum_ld: h = x +
 *                      residual, the residual stream behind this place; only with a
 *                      residual. It may be residual itself, or x where the types are
 *                      the same (same address and stride)
 *   sum_dtype          `dtype`, or ZS_F32 with bf16 x; read only with a residual
 *   weight[dim]        DEVICE, `wdtype` (ZS_F32 or ZS_BF16), or NULL (ones)
 *   eps                finite in fp32, >= 0
 *   y[rows, dim]       DEVICE, `dtype`, row stride y_ld: y = h * rstd * weight with
 *                      rstd = 1 / sqrt(sum(h^2) / dim + eps), of h before it is
 *                      rounded; NULL (skip) only with codes
 *   codes[rows, dim], scales[rows, ceil(dim / 128)]
 *                      optional DEVICE (both or none): y in 8 bits, as
 *                      zs_activation_pack gives it for y before its rounding
 *   rstd[rows]         optional DEVICE fp32 (the backward pass needs it)
 * Apart from sum in place no output may share bytes with another argument.
 * Any finite h of any size gives the norm of that formula: where the sum of squares
 * leaves fp32's range, it is made again of h times a power of two (rstd is subnormal for
 * root mean squares above 2^126, and infinite for those below 2^-128 with eps 0, or of
 * zeros). Errors: ZS_ERR_NULL (sum without residual, neither y nor codes, codes or scales alone
 * among them), ZS_ERR_SIZE (dim < 1 with rows > 0 among them), ZS_ERR_DTYPE,
 * ZS_ERR_HPARAM, ZS_ERR_ALIGN, ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_rms_norm_forward(const void* x, int32_t dtype, int64_t x_ld, const void* residual,
                              int64_t residual_ld, void* sum, int64_t sum_ld, int32_t sum_dtype,
                              const void* weight, int32_t wdtype, int64_t rows, int64_t dim, double eps,
                              void* y, int64_t y_ld, uint8_t* codes, int64_t codes_ld, float* scales,
                              int64_t scales_ld, float* rstd, hipStream_t stream);

/* Bytes of workspace zs_rms_norm_backward needs for the weight's gradient (0 for
 * sizes it refuses). The contents need no initialisation. */
size_t zs_rms_norm_workspace_bytes(int64_t rows, int64_t dim);

/*
 * zs_rms_norm_backward -- gradients of the RMS norm.
 *   dy[rows, dim]      DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride dy_ld
 *   h[rows, dim]       DEVICE, what was normed (sum, or x without a residual), row
 *                      stride h_ld: `dh_dtype`, or ZS_E4M3 codes with
 *   scales[rows, ceil(dim / 128)]
 *                      DEVICE fp32, row stride scales_ld, read only with codes
 *   weight[dim]        DEVICE, `wdtype`, or NULL (ones)
 *   rstd[rows]         DEVICE fp32, as zs_rms_norm_forward gives it
 *   dres[rows, dim]    optional DEVICE (NULL = none), `dh_dtype`, row stride dres_ld:
 *                      the gradient that reaches h along the residual stream
 *   dh[rows, dim]      DEVICE, `dh_dtype` (`dtype`, or ZS_F32 with bf16 dy), row
 *                      stride dh_ld: with xh = h * rstd,
 *                      dh = rstd * (dy * weight - xh * mean(dy * weight * xh)) + dres,
 *                      the gradient of x and of the residual alike; it may be dres
 *                      itself (same address and stride)
 *   dweight[dim]       optional DEVICE, `grad_dtype`:
 *                      (first ? 0 : dweight) + sum over rows of dy * xh
 *   workspace          DEVICE scratch of at least zs_rms_norm_workspace_bytes(rows,
 *                      dim) bytes on a 16-byte boundary, required unless dweight is
 *                      NULL or there are no rows; calls and graph replays that may run
 *                      at the same time need one each
 * rows == 0 with first != 0 sets dweight to zero. Apart from dh in place no output
 * may share bytes with an input, the workspace or another output. Errors:
 * ZS_ERR_NULL, ZS_ERR_SIZE, ZS_ERR_DTYPE, ZS_ERR_WORKSPACE, ZS_ERR_ALIGN,
 * ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_rms_norm_backward(const void* dy, int32_t dtype, int64_t dy_ld, const void* h,
                               int32_t h_dtype, int64_t h_ld, const float* scales, int64_t scales_ld,
                               const void* weight, int32_t wdtype, const float* rstd, const void* dres,
                               int64_t dres_ld, int64_t rows, int64_t dim, void* dh, int64_t dh_ld,
                               int32_t dh_dtype, void* dweight, int32_t grad_dtype, int32_t first,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that the two calls below need for n tokens over [vocab, dim],
 * with hidden states and weight of `dtype`: zs_linear_cross_entropy_backward with
 * a dweight of `grad_dtype`, or, with grad_dtype -1, zs_linear_cross_entropy_forward
 * (0 for sizes and types that they refuse). The contents need no initialisation. */
size_t zs_linear_cross_entropy_workspace_bytes(int64_t n, int64_t vocab, int64_t dim, int32_t dtype,
                                               int32_t grad_dtype);

/*
 * zs_linear_cross_entropy_forward -- softmax cross entropy of the logits
 * z = hidden weight^T over the vocabulary, without keeping the logits.
 *   hidden[n, dim]     DEVICE, `dtype` (ZS_F32 or ZS_BF16), row stride hidden_ld
 *   weight[vocab, dim] DEVICE, `dtype`, row stride weight_ld: the head, or the
 *                      embedding's table where they are tied
 *   labels[n]          DEVICE ids, `index_type` ZS_I32 or ZS_I64; a token whose
 *                      label is outside of [0, vocab) does not count
 *   loss[n]            DEVICE fp32: log(sum_v exp(z_v)) - z_label, 0 where a
 *                      token does not count
 *   lse[n]             optional DEVICE fp32 (NULL = skip; the backward pass needs
 *                      it): log(sum_v exp(z_v)), 0 where a token does not count
 *   workspace          DEVICE scratch of at least
 *                      zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, dtype, -1)
 *                      bytes on a 16-byte boundary; calls and graph replays that
 *                      may run at the same time need one each
 * Products of bf16 values are exact and added in fp32. fp32 values enter as they
 * are for up to 64 tokens, as sums of two fp16 scaled by a power of two of their row
 * for more: a product h w is off by up to 2^-20 |h w|, or 2^-39 of one's magnitude by
 * the largest of the other's row. Infinite or NaN logits make their token's loss
 * infinite or NaN, and no other's; one of minus infinity counts as 0 (in fp32 over more than 64
 * tokens an infinite value times one below 2^-39 of its row's largest is NaN, as times 0). n and vocab are
 * below 2^31, dim at most 2^20, with at most 2^31 - 1 tiles of 128 rows of the head
 * by 128 tokens. Weights that lie on 16-byte boundaries with a multiple of 64 columns
 * are read as they lie; others are laid out in the workspace first. No output or
 * workspace may share bytes with another argument. Errors: ZS_ERR_NULL, ZS_ERR_SIZE
 * (dim < 1 with n > 0 among them), ZS_ERR_DTYPE, ZS_ERR_WORKSPACE, ZS_ERR_ALIGN,
 * ZS_ERR_OVERLAP, ZS_ERR_HIP.
 */
zs_status zs_linear_cross_entropy_forward(const void* hidden, int64_t hidden_ld, int32_t dtype,
                                          const void* weight, int64_t weight_ld, const void* labels,
                                          int32_t index_type, int64_t n, int64_t vocab, int64_t dim,
                                          float* loss, float* lse, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream);

/*
 * zs_linear_cross_entropy_backward -- gradients of that loss. With
 * g_iv = scale * dloss_i * (exp(z_iv - lse_i) - [v == label_i]), 0 for tokens
 * that do not count:
 *   hidden, weight, labels
 *                      as above; lse[n] as the forward pass gives it
 *   dloss[n]           optional DEVICE fp32 gradient of each token's loss (NULL =
 *                      ones); scale must be finite (1 / tokens for a mean)
 *   dhidden[n, dim]    DEVICE, `dtype`, row stride dhidden_ld: sum_v g_iv weight_v,
 *                      zeros where a token does not count
 *   dweight[vocab, dim]
 *                      DEVICE, `grad_dtype`, row stride dweight_ld:
 *                      (first ? 0 : dweight) + sum_i g_iv hidden_i; hidden states
 *                      of tokens that do not count reach no sum, whatever they hold
 *   workspace          DEVICE scratch of at least
 *                      zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, dtype,
 *                      grad_dtype) bytes on a 16-byte boundary; calls and graph
 *                      replays that may run at the same time need one each
 * The logits are made again, a piece of the vocabulary at a time, of fp32 values as
 * sums of three bf16 for up to 511 tokens, with an error of the size of fp32 products'
 * roundings, and of two fp16 as above for more. An
 * infinite value makes the gradients that it reaches NaN. g is rounded to bf16 for
 * the gradients that are stored in bf16 from bf16 inputs, and has 24 bits for the
 * others; sums are fp32, in an order that depends on the sizes and on how many tokens
 * count alone. n == 0 with first != 0 sets dweight to zero.
 * Limits, overlaps and errors as above, and ZS_ERR_HPARAM.
 */
zs_status zs_linear_cross_entropy_backward(const void* hidden, int64_t hidden_ld, int32_t dtype,
                                           const void* weight, int64_t weight_ld, const void* labels,
                                           int32_t index_type, const float* lse, const float* dloss,
                                           float scale, int64_t n, int64_t vocab, int64_t dim,
                                           void* dhidden, int64_t dhidden_ld, void* dweight,
                                           int32_t grad_dtype, int64_t dweight_ld, int32_t first,
                                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Static, NUL-terminated name of a status code ("ZS_OK", "ZS_ERR_NULL", ...). */
const char* zs_status_string(zs_status status);

/* Library version as major*10000 + minor*100 + patch. */
int32_t zs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZS_H_ */
