/*
 * gemma_nq -- fused residual add + Gemma RMSNorm + next-linear input
 * quantization on one GB300 (sm_103a), as a C ABI.
 *
 * The operation ("vllm.models.qwen3_5.nvidia.ops.fused_norm_quant", module
 * docstring and gemma_add_rms_norm_quant):
 *
 *     h  = x + residual                 (rounded to the activation dtype;
 *                                        written back into `residual`)
 *     y  = dtype(h * rsqrt(mean(h^2) + eps) * (1 + w))
 *     q  = quant(y)                     (computed from the rounded y)
 *
 * with quant one of
 *   GNQ_FP8   static per-tensor FP8 E4M3: q = e4m3_satfinite(y / scale);
 *   GNQ_NVFP4 per 16-element block: E4M3 block scale
 *             sf = e4m3_satfinite(g * (amax / 6)), codes
 *             e2m1_satfinite(y * (g / sf)) packed two per byte, the
 *             lower-indexed element in the low nibble; block scales in the
 *             128x4 swizzled layout of shape (round_up(M,128),
 *             round_up(H/16,4)), byte (m, b) at
 *             ((m/128)*(Kp/4) + b/4)*512 + (m%32)*16 + ((m%128)/32)*4 + b%4;
 *   GNQ_MXFP8 per 32-element block ("vllm.model_executor.layers.
 *             fused_allreduce_gemma_rms_norm", allreduce_gemma_rms_norm_mxfp8):
 *             E8M0 scale code floor(log2(amax)) - 8 + 127 clamped to
 *             [0, 254] (0 for an all-zero block), stored row-major (M, H/32);
 *             codes e4m3_satfinite(y / 2^(code - 127)).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are addresses the current CUDA device can access,
 *    in row-major contiguous layout: device memory, or pinned host memory
 *    (mapped into the device's address space; on a Grace-Blackwell node the
 *    kernels then read and write it over NVLink-C2C, with no separate copy).
 *    A call whose activations are not in device memory always runs one CTA
 *    per row (plain loads and stores), never the streaming kernel, whose
 *    bulk copies read device memory.  Activations x, residual, y and the weight
 *    w are 16-bit, of the type named by `dtype` (GNQ_BF16 or GNQ_FP16).
 *  - The caller owns and allocates every buffer.  The library allocates
 *    nothing per call and keeps no state other than cached device properties.
 *  - x, w, scale and the partial buffers are read only.  `residual` (when not
 *    NULL) is updated in place to the rounded x + residual.  q, block_scale
 *    and y are written.  Rows m >= M of the NVFP4 scale tensor are NOT
 *    written (their bytes keep whatever the caller put there).
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream).  Nothing is synchronised and no host copy is made.
 *  - M == 0 returns GNQ_OK without launching anything.
 *  - Every call returns a gnq_status; the library never aborts, exits or
 *    traps.  Argument checks happen before any launch; a rejected call has
 *    no effect.
 *  - Alignment: x, residual, w, y, q and every partial buffer must be 16-byte
 *    aligned, block_scale 4-byte aligned, scale 4-byte aligned
 *    (GNQ_ERR_ALIGN).  NVFP4 calls whose 16-bit tensors (and partial
 *    stride) are also 32-byte aligned, as every allocator's tensors are,
 *    move each 16-element block in one 256-bit access; others run one CTA
 *    per row with 128-bit accesses.  H must be a multiple of 8 (GNQ_ERR_SHAPE); NVFP4 needs
 *    H % 64 == 0 (whole 4-column scale tiles, so padded scale columns never
 *    exist) and MXFP8 H % 32 == 0.  H is at most 65536.
 *  - x and residual must not be the same buffer, and y must differ from both
 *    (GNQ_ERR_ALIAS).  gemma_sandwich_norm_quant, gnq_quantize,
 *    gated_act_quant, gnq_nvfp4_dequantize, nvfp4_linear and the entry points
 *    of a mixture of experts check whole ranges: what such a call writes may
 *    share no byte with what it reads (but residual_out may be `residual`
 *    itself, and out of gnq_expert_combine its `add`) nor with another output.
 *  - Every buffer must hold at least the elements its shape below states;
 *    the library receives raw pointers and cannot check sizes (the Python
 *    binding does, before any launch).
 */
#ifndef GEMMA_NQ_H
#define GEMMA_NQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GNQ_OK = 0,
    GNQ_ERR_NULL = 1,  /* a required pointer is NULL                        */
    GNQ_ERR_SHAPE = 2, /* M < 0, H out of range or not a supported multiple */
    GNQ_ERR_DTYPE = 3, /* dtype is not GNQ_BF16 / GNQ_FP16                  */
    GNQ_ERR_MODE = 4,  /* unknown quantization mode, or k out of range      */
    GNQ_ERR_ALIAS = 5, /* x == residual, or y aliases x or residual         */
    GNQ_ERR_ALIGN = 6, /* a pointer or the partial stride is misaligned     */
    GNQ_ERR_CUDA = 7,  /* the CUDA runtime reported an error at launch (the
                          runtime's last-error state is cleared, so the
                          caller's own later checks do not see it)         */
    GNQ_ERR_MEMORY = 8 /* a buffer that must be in the current device's
                          memory is not                                    */
} gnq_status;

/* Activations are GNQ_BF16 or GNQ_FP16; GNQ_FP32 and GNQ_E4M3 are further
 * output types of nvfp4_linear and gnq_nvfp4_dequantize. */
typedef enum { GNQ_BF16 = 0, GNQ_FP16 = 1, GNQ_FP32 = 2, GNQ_E4M3 = 3 } gnq_dtype;

typedef enum { GNQ_FP8 = 0, GNQ_NVFP4 = 1, GNQ_MXFP8 = 2 } gnq_mode;

typedef enum { GNQ_SILU = 1, GNQ_GELU_TANH = 2 } gnq_act;

/*
 * Residual add + Gemma RMSNorm, no quantization
 * ("vllm.model_executor.layers.fused_allreduce_gemma_rms_norm",
 * fused_allreduce_gemma_rms_norm: at tensor-parallel size 1 it is
 * norm(hidden_states, residual), returning (normed, new residual)).
 *
 *   x        (M, H) activation, read only.
 *   residual (M, H) or NULL; updated in place to dtype(x + residual).
 *   w        (H,) Gemma weight; the norm multiplies by (1 + w).
 *   eps      RMSNorm epsilon.
 *   y        (M, H) output, y = dtype(h * rsqrt(mean(h^2) + eps) * (1 + w)).
 */
int gemma_add_rms_norm(const void *x, void *residual, const void *w, float eps,
                       void *y, int64_t M, int64_t H, int dtype, void *stream);

/*
 * Residual add + Gemma RMSNorm + the next linear's input quantization, in one
 * pass ("vllm.models.qwen3_5.nvidia.ops.fused_norm_quant",
 * gemma_add_rms_norm_quant).
 *
 *   x, residual, w, eps   as for gemma_add_rms_norm.
 *   scale        device pointer to ONE fp32: the static FP8 scale s, or the
 *                NVFP4 global scale g (input_global_scale_inv).  Read on the
 *                device, so it may change between graph replays.  Unused
 *                (may be NULL) for GNQ_MXFP8.
 *   mode         GNQ_FP8, GNQ_NVFP4 or GNQ_MXFP8.
 *   write_y      nonzero: also store the normed activation y (M, H).
 *   q            FP8 / MXFP8: (M, H) E4M3 codes.  NVFP4: (M, H/2) bytes of
 *                packed E2M1 codes.
 *   block_scale  NVFP4: the swizzled (round_up(M,128), round_up(H/16,4))
 *                E4M3 scale bytes.  MXFP8: (M, H/32) E8M0 codes.  Unused
 *                (may be NULL) for GNQ_FP8, whose block scale is `scale`.
 *   y            (M, H) if write_y, else ignored (may be NULL).
 */
int gemma_add_rms_norm_quant(const void *x, void *residual, const void *w,
                             float eps, const float *scale, int mode,
                             int write_y, void *q, void *block_scale, void *y,
                             int64_t M, int64_t H, int dtype, void *stream);

/*
 * As gemma_add_rms_norm_quant, with the activation given as k partial
 * buffers, the per-rank partial outputs of a row-parallel linear that a
 * tensor-parallel all-reduce would sum ("vllm.models.qwen3_5.nvidia.ops.
 * fused_allreduce_norm_quant", fused_allreduce_gemma_rms_norm_quant:
 * hidden_states is the per-rank partial, reduced with fp32 accumulation).
 * Here the k partials sit in this GPU's memory and are summed locally:
 * a = dtype(((p0 + p1) + p2) + ...) in fp32, then h = dtype(a + residual).
 *
 *   x_parts      base of k (M, H) buffers; partial p starts at
 *                x_parts + p * part_stride ELEMENTS (part_stride >= M*H and a
 *                multiple of 8, so every partial is 16-byte aligned).
 *   k            number of partials, 1..8 (GNQ_ERR_MODE otherwise).
 *   mode         as above, or -1 for no quantization (then write_y must be
 *                nonzero and q / block_scale / scale are ignored).
 */
int gemma_add_rms_norm_quant_parts(const void *x_parts, int k,
                                   int64_t part_stride, void *residual,
                                   const void *w, float eps,
                                   const float *scale, int mode, int write_y,
                                   void *q, void *block_scale, void *y,
                                   int64_t M, int64_t H, int dtype,
                                   void *stream);

/*
 * Plain (non-Gemma) RMSNorm variant: y = dtype(h * rsqrt(mean(h^2) + eps) * w),
 * i.e. weight bias 0 instead of 1 ("vllm.models.qwen3_5.nvidia.ops.
 * fused_allreduce_norm_quant" passes the weight bias to the fused kernel;
 * weight_bias=1.0 marks the Gemma form on
 * "vllm.model_executor.layers.fused_allreduce_gemma_rms_norm").  Arguments
 * as for gemma_add_rms_norm_quant_parts; k = 1 for a single activation.
 */
int add_rms_norm_quant(const void *x_parts, int k, int64_t part_stride,
                       void *residual, const void *w, float eps,
                       const float *scale, int mode, int write_y, void *q,
                       void *block_scale, void *y, int64_t M, int64_t H,
                       int dtype, void *stream);

/*
 * Sandwich norm: the norm after a block, its gate and residual scale, the
 * residual add, and the norm before the next block with the quantization for
 * that block's first linear, in one pass:
 *
 *     u = x * rsqrt(mean(x^2) + eps) * (1 + w_post)    (u = x if w_post is NULL)
 *     h = dtype(residual + residual_scale * gate * u)  (one rounding; gate 1 if NULL)
 *     y = dtype(h * rsqrt(mean(h^2) + eps) * (1 + w))
 *     q = quant(y)
 *
 *   x            (M, H) the block's output, read only.
 *   residual     (M, H), required.
 *   residual_out (M, H) receives h; NULL or `residual` itself: updated in
 *                place.
 *   w_post, w    (H,) Gemma weights; w_post may be NULL.
 *   gate         NULL, (H,) with gate_stride 0 (one gate per channel), or
 *                (M, H) with rows gate_stride elements apart (>= H, a multiple
 *                of 8); of the activation type, 16-byte aligned.
 *   mode, write_y, scale, q, block_scale, y   as for
 *                gemma_add_rms_norm_quant_parts (mode -1: y only).
 * A row of more than 8192 elements (NVFP4: 16384) is split evenly over 2, 4 or
 * 8 CTAs, in multiples of 8 elements (MXFP8: 32, NVFP4: 64); an H that does
 * not divide so is GNQ_ERR_SHAPE.
 */
int gemma_sandwich_norm_quant(const void *x, void *residual,
                              void *residual_out, const void *w_post,
                              const void *w, const void *gate,
                              int64_t gate_stride, float residual_scale,
                              float eps, const float *scale, int mode,
                              int write_y, void *q, void *block_scale, void *y,
                              int64_t M, int64_t H, int dtype, void *stream);

/*
 * Quantization of a 16-bit matrix: q = quant(x), the codes and scales that
 * the norm entry points give for a y equal to x.
 *   x          (M, H), rows row_stride elements apart (>= H, a multiple of 8).
 *   scale, mode, q, block_scale   as for gemma_add_rms_norm_quant.
 */
int gnq_quantize(const void *x, int64_t row_stride, const float *scale,
                 int mode, void *q, void *block_scale, int64_t M, int64_t H,
                 int dtype, void *stream);

/*
 * The gated activation between the products of an MLP, and the quantization
 * for the second: y = dtype(act(gate) * up) in fp32, rounded once; q = quant(y).
 * (Before that rounding act(gate) * up is good to 5e-6 of its value while
 * act(gate) is above 1e-4 of the gate, to 7e-5 below; an act(gate) below 2^-218
 * gives 0.)
 *   x          (M, 2H): gate in the first H columns, up in the last; rows
 *              row_stride elements apart (>= 2H, a multiple of 8).
 *   act        GNQ_SILU: g / (1 + exp(-g)); GNQ_GELU_TANH: g/2 (1 + tanh(
 *              sqrt(2/pi) (g + 0.044715 g^3))).
 *   mode, write_y, scale, q, block_scale, y   as for
 *              gemma_add_rms_norm_quant_parts (mode -1: y only).
 */
int gated_act_quant(const void *x, int64_t row_stride, int act,
                    const float *scale, int mode, int write_y, void *q,
                    void *block_scale, void *y, int64_t M, int64_t H,
                    int dtype, void *stream);

/*
 * NVFP4 codes and swizzled block scales back to plain values:
 * out = type(code * (block scale / g)), the quotient and the product each
 * rounded to fp32.
 *   scale      device pointer to the global scale g, or NULL for 1.
 *   out        (M, K) of out_type GNQ_BF16, GNQ_FP16, GNQ_FP32, or GNQ_E4M3
 *              (saturating).
 */
int gnq_nvfp4_dequantize(const void *q, const void *block_scale,
                         const float *scale, void *out, int64_t M, int64_t K,
                         int out_type, void *stream);

/*
 * Product of an NVFP4 activation with an NVFP4 weight:
 *
 *     y[m, n] = type(alpha * sum_k a[m, k] w[n, k] + bias[n])
 *
 * a and w being the codes times their block scales (products exact, sums in
 * fp32), alpha usually 1 / (global scale of a * global scale of w).
 *   q, block_scale      (M, K/2) packed codes and the swizzled scales of the
 *                       activation, as the NVFP4 mode of the other entry
 *                       points writes them; scale rows m >= M are read but
 *                       affect nothing.
 *   w_q, w_block_scale  (N, K/2) and the swizzled (round_up(N,128), K/16)
 *                       scales of the weight, one row per output.
 *   alpha               device pointer to ONE fp32.
 *   bias                (N,) or NULL; of bias_type GNQ_BF16 or GNQ_FP16,
 *                       which must be out_type unless that is GNQ_FP32.
 *   y                   (M, N) of out_type GNQ_BF16, GNQ_FP16 or GNQ_FP32.
 * K is a multiple of 64, at most 65536; M and N are any sizes.  The codes,
 * block scales and y must be in the current device's memory (GNQ_ERR_MEMORY)
 * and 16-byte aligned.
 */
int nvfp4_linear(const void *q, const void *block_scale, const void *w_q,
                 const void *w_block_scale, const float *alpha,
                 const void *bias, void *y, int64_t M, int64_t N, int64_t K,
                 int out_type, int bias_type, void *stream);

/*
 * Mixture of experts.  The five entry points below share one order of rows,
 * by expert: expert e owns rows offsets[e] .. offsets[e + 1] - 1 of the R rows
 * that a buffer holds; offsets are E + 1 int32 on the device, ascending from 0
 * to at most R, and are never read on the host.  Rows from offsets[E] on belong
 * to nobody: what they hold influences nothing, and what is written leaves them
 * as they were.
 * Block scales keep the 128x4 layout, each expert's rows starting a 128-row
 * tile of their own, tile offsets[e] / 128 + e (rounded down): a buffer of
 * R / 128 + E tiles of 128 rows holds any split.  Bytes of a tile beyond an
 * expert's last row are not written and influence nothing.
 * 1 <= E <= 1024 and 1 <= k <= 32.  scale_stride (alpha_stride) is 1 for one
 * fp32 per expert, 0 for one that all share (GNQ_ERR_MODE otherwise).
 * Offsets that do not ascend from 0 to at most R, and slots that are not a row
 * of their expert, are found on the device by each call that has rows: bit 2 of
 * the device error word is set (gnq_read_device_error) and nothing outside the
 * buffers is touched.  Of such offsets nvfp4_expert_linear writes nothing at
 * all; the quantization and the way back leave out rows that no expert's bounds
 * hold and slots that are no row of their expert, and give each other row to an
 * expert whose bounds hold it.
 */

/*
 * The router: the k largest logits of each token and their softmax weights,
 * and the rows of the chosen experts.
 *
 *   logits      (M, E) of logits_type GNQ_BF16, GNQ_FP16 or GNQ_FP32 (exact in
 *               fp32, compared there), rows row_stride >= E elements apart,
 *               aligned to their size.
 *   experts     (M, k) int32: by falling logit, equal logits by rising index,
 *               NaN above every number.  A logit of -inf is never chosen:
 *               where only such are left, expert and slot are -1 and the
 *               weight is 0 (a token of a padded batch has -inf alone).
 *   weights     (M, k) fp32: scale * exp(l_j - l_0) / sum, the sum over the
 *               chosen (renormalize nonzero) or over all E logits.  A NaN or
 *               +inf among the summed logits makes the token's weights NaN.
 *   offsets     (E + 1) int32, written; offsets[E] is the number of rows.
 *   slots       (M, k) int32: the row of (t, j).  An expert's rows are in
 *               token order.
 * M may be 0 (the offsets are then 0); k <= E; M * k <= 2^31 - 2^16.
 */
int gnq_expert_route(const void *logits, int64_t row_stride, int logits_type,
                     int64_t M, int64_t E, int k, int renormalize, float scale,
                     int32_t *experts, float *weights, int32_t *offsets,
                     int32_t *slots, void *stream);

/*
 * Rows to NVFP4 with the global scale of their expert, in expert order.
 *   x           (M, H), or (M, 2H) with act, rows row_stride elements apart as
 *               for gnq_quantize and gated_act_quant.
 *   act         0: y = x; GNQ_SILU, GNQ_GELU_TANH: y = dtype(act(gate) * up) as
 *               gated_act_quant computes it.
 *   slots, experts  (M, k) as gnq_expert_route gives them: y[t] goes to every
 *               row slots[t, j] (those below 0 are dropped).  Two slots must
 *               not name the same row.  Both NULL: x is in expert order
 *               already, M equals R, and k is ignored.
 *   scale       global scale(s) g.
 *   q           (R, H/2) packed codes.
 *   block_scale (R / 128 + E) * 128 rows of H/16 scale bytes.
 * H is a multiple of 64.
 */
int gnq_expert_quantize(const void *x, int64_t row_stride, int act,
                        const int32_t *offsets, int64_t E, const int32_t *slots,
                        const int32_t *experts, int k, const float *scale,
                        int scale_stride, void *q, void *block_scale, int64_t R,
                        int64_t M, int64_t H, int dtype, void *stream);

/*
 * The way back: out = type(code * (block scale / g)) as gnq_nvfp4_dequantize,
 * for rows in expert order.  scale may be NULL (1).
 */
int gnq_expert_dequantize(const void *q, const void *block_scale,
                          const int32_t *offsets, int64_t E, const float *scale,
                          int scale_stride, void *out, int64_t R, int64_t K,
                          int out_type, void *stream);

/*
 * Products grouped by expert: row r of expert e gives
 *
 *     y[r, n] = type(alpha[e] * sum_k a[r, k] w[e, n, k] + bias[e, n])
 *
 *   q, block_scale  the activation, as gnq_expert_quantize writes it.
 *   w_q             (E, N, K/2) packed codes.
 *   w_block_scale   E times the swizzled (round_up(N,128), K/16) scales of one
 *                   expert's weight, as gnq_quantize writes them.
 *   alpha           device fp32, usually 1 / (scale of a * scale of w).
 *   bias            (E, N) or NULL, of bias_type, as for nvfp4_linear.
 *   y               (R, N) of out_type GNQ_BF16, GNQ_FP16 or GNQ_FP32.
 * K is a multiple of 64, at most 65536; N is any size, N * E < 2^28.  Memory
 * and alignment as for nvfp4_linear.
 */
int nvfp4_expert_linear(const void *q, const void *block_scale, const void *w_q,
                        const void *w_block_scale, const float *alpha,
                        int alpha_stride, const void *bias,
                        const int32_t *offsets, int64_t E, void *y, int64_t R,
                        int64_t N, int64_t K, int out_type, int bias_type,
                        void *stream);

/*
 * The weighted sum of a token's rows:
 *
 *     out[t] = type(sum_j weights[t, j] * y[slots[t, j]] + add[t])
 *
 * in fp32, two neighbours at a time in the order of j, `add` last, rounded
 * once: the same bits whatever else the batch holds.  Slots below 0 add
 * nothing; a slot of R or more is reported as above and adds nothing.
 *   y        (R, H) of y_type GNQ_BF16, GNQ_FP16 or GNQ_FP32.
 *   weights  (M, k) fp32.
 *   add      (M, H) of out_type or NULL; may be `out` itself.
 *   out      (M, H) of out_type: y_type, or any of the three if that is GNQ_FP32.
 * H is a multiple of 8.
 */
int gnq_expert_combine(const void *y, const int32_t *slots, const float *weights,
                       const void *add, void *out, int64_t R, int64_t M,
                       int64_t H, int k, int y_type, int out_type, void *stream);

/* Human-readable text of a gnq_status (static storage, never NULL). */
const char *gnq_status_string(int status);

/*
 * Tuning hook: force the launch shape of later calls in this process.
 *   kernel   0 = automatic; 1 = one CTA (or cluster) per row; 2 = persistent
 *            streaming kernel (rows staged through shared memory).
 *   cluster  row kernel: 0 = automatic, else 1, 2, 4 or 8 CTAs per row.
 *            Streaming kernel: 0 = automatic grid, else at least that many
 *            rows (2, 4 or 8) per CTA (grid = ceil(M / cluster) CTAs when
 *            that is below one wave).
 *   vpt      0 = automatic, else 1, 2 or 4 units (8 elements; 16 for
 *            NVFP4) per thread.
 *   form     0 = automatic; 1 = h and the weight unpacked to fp32 (fewest
 *            instructions); 2 = kept packed (fewest registers; Gemma or plain
 *            weight bias only).
 * A forced shape that does not fit a call (H, mode, shared memory) falls back
 * to the automatic one for that call.  The shape only changes the order in
 * which a row's squares are summed (so y may move by one rounding step); the
 * residual, and the codes of a given y, never depend on it.  Not
 * synchronised with calls in flight on other host threads.  Returns
 * GNQ_ERR_SHAPE for values outside those sets.
 */
int gnq_set_launch_policy(int kernel, int cluster, int vpt, int form);

/*
 * The launch shape the automatic policy picks for a call on the current
 * device with its activations in device memory, in the terms of
 * gnq_set_launch_policy (a forced policy is not applied): *kernel 1 or 2, *cluster CTAs per row (0 for the streaming
 * kernel), *vpt 1, 2 or 4, *form 1 (fp32) or 2 (packed).  The arguments
 * describe the call: rows M >= 1, width H, k partial buffers (1: one
 * activation), whether it has a residual and writes y, mode, dtype, and the
 * weight bias (1 Gemma, 0 plain).  Forcing the returned shape reproduces
 * the automatic launch, for instance to run a call that writes y with
 * exactly the arithmetic of one that does not.  Returns GNQ_OK;
 * GNQ_ERR_NULL, GNQ_ERR_DTYPE, GNQ_ERR_MODE or GNQ_ERR_SHAPE for arguments a
 * call would reject; GNQ_ERR_CUDA without a usable device.
 */
int gnq_query_launch(int64_t M, int64_t H, int k, int has_residual, int write_y, int mode,
                     int dtype, float weight_bias, int *kernel, int *cluster, int *vpt,
                     int *form);

/*
 * Tuning hook: force the kernel of later nvfp4_linear and nvfp4_expert_linear
 * calls in this process.  kernel 0 = automatic; 1 = tiles of one CTA
 * (nvfp4_linear: K split over a cluster where that fills the device); 2 = CTA
 * pairs on 256 x 256 tiles.  (More tiles of nvfp4_linear than a grid holds go to
 * pairs all the same.)  A split adds its parts last, so y may
 * move by a rounding step of the fp32 sum.  Not synchronised with calls in
 * flight on other host threads.  Returns GNQ_ERR_SHAPE for other values.
 */
int gnq_set_linear_policy(int kernel);

/*
 * The kernel that nvfp4_linear picks by itself for a shape on the current
 * device, in the terms of gnq_set_linear_policy (a forced one is not applied):
 * *kernel 1 or 2, *tokens the tokens of a tile, *split the CTAs that share a
 * tile's K.  M >= 1.  Returns GNQ_OK; GNQ_ERR_NULL, GNQ_ERR_DTYPE or
 * GNQ_ERR_SHAPE for arguments that a call would reject; GNQ_ERR_CUDA without a
 * usable device.
 */
int gnq_query_linear(int64_t M, int64_t N, int64_t K, int out_type, int *kernel, int *tokens, int *split);

/*
 * Programmatic dependent launch (on by default): each launch may start while
 * the preceding kernel on the stream drains, and waits inside the kernel
 * (griddepcontrol.wait) until that kernel's results are visible before its
 * first global read of them.  Before the wait, the CTAs that can be waiting
 * (the first wave of a one-CTA-per-row launch; streaming CTAs, for their
 * first rows, in the NVFP4, MXFP8 and bf16 instances) prefetch their rows
 * of x, the partials and the residual
 * into L2: a cache hint, not a read (the values used are loaded after the
 * wait, and L2 is where the preceding kernel's stores land), so the
 * buffers must be valid device-accessible memory at launch, as for any
 * call.  Right after the wait the kernel also lets a programmatic
 * dependent that follows it launch (that kernel must wait in the same way
 * before reading these outputs), so the dependent's CTAs can take the SMs
 * this grid leaves idle and run their own prologue early.  Results are
 * identical either way.  enable = 0 turns it off for later calls in this
 * process, 1 turns it on.  Not synchronised with calls in flight on other
 * host threads.
 */
int gnq_set_pdl(int enable);

/*
 * Constant weights (off by default).  With enable = 1, later small-batch
 * calls (those the policy runs one 16-byte unit -- NVFP4: one 16-element
 * block -- per thread on the one-CTA-per-row kernel, i.e. batches below about
 * one row per SM, with one activation rather than partials) read the norm
 * weight w and the quantization scale, and build their quantizer constants,
 * before they wait for the preceding kernel on their stream (programmatic
 * dependent launch), so that work overlaps its tail; so do nvfp4_linear calls
 * that run on tiles of at most 128 tokens with the first part of the weight's
 * codes and block scales.  Other calls ignore the flag.  The caller
 * guarantees that no kernel that precedes a call on its stream, and may still
 * be running, writes w, the scale, or the linear's weight (true when they are
 * model constants).  x, the partials, the residual and the linear's
 * activation are always read after the wait.  Results are identical either
 * way.  enable = 0 restores the default.  Not synchronised with calls in
 * flight on other host threads.
 * Returns GNQ_ERR_SHAPE for other values.
 */
int gnq_set_constant_weights(int enable);

/*
 * Test hook for the failure path of the bounded waits (off by default).
 * With enable = 1, later launches of the persistent streaming kernel, of
 * nvfp4_linear and of nvfp4_expert_linear in this process announce 16 bytes more per row (per stage of
 * K) than their copies deliver and give a wait at most ~2^20 clock cycles, so
 * each CTA's wait for its first row (stage) gives up: the kernel sets bit 1
 * of the device error word, completes each outstanding barrier with one more
 * valid 16-byte copy (from w, or the weight's block scales, into its own
 * shared memory, so every copy has landed before it returns), and returns
 * without writing any output.  Nothing outside the call's own buffers is
 * touched; the other kernels are unaffected.  enable = 0 restores normal
 * launches.  Not synchronised with calls in flight on other host threads.
 * Returns GNQ_ERR_SHAPE for other values.
 */
int gnq_inject_wait_timeout(int enable);

/*
 * Test hook for a split product that loses one part (off by default, cta =
 * -1).  With cta = 0..7, later launches of nvfp4_linear that share a tile's K
 * among several CTAs (a cluster) make that CTA of each cluster alone give up, in
 * the way gnq_inject_wait_timeout does; bit 1 of the device error word is set
 * and no CTA of the cluster writes output.  Launches without such a CTA are
 * unaffected.  Not synchronised with calls in flight on other host threads.
 * Returns GNQ_ERR_SHAPE for other values.
 */
int gnq_inject_split_timeout(int cta);

/*
 * Device error word of the current device.  Every wait inside a kernel is
 * bounded; a kernel whose wait gives up (about a second without progress)
 * skips the rest of its work, sets bit 1 here and returns, leaving its
 * outputs incomplete.  Bit 2: an entry point of a mixture of experts met
 * offsets or slots that name no row.  Copies the word into *flags (synchronising the device)
 * and clears it when `clear` is nonzero.
 */
int gnq_read_device_error(unsigned int *flags, int clear);

/*
 * Diagnostic: a stand-in for the first kernel of the next linear layer, to
 * measure programmatic dependent launch with a real consumer.  Launched as a
 * programmatic dependent of the preceding kernel on `stream`, with `ctas`
 * CTAs of 256 threads: each CTA first reads its share of the wt_bytes at
 * `wt` (an independent buffer, standing for the layer's weight), then waits
 * for the preceding kernel's results (griddepcontrol.wait), then reads its
 * share of the q_bytes at `q` (that kernel's codes), and stores one checksum
 * word per thread to `out` (ctas * 256 words).  Byte counts are multiples of
 * 16 and the pointers 16-byte aligned device memory.  Returns GNQ_ERR_SHAPE,
 * GNQ_ERR_NULL or GNQ_ERR_CUDA on bad arguments or a failed launch.
 */
int gnq_pdl_consumer(const void *q, int64_t q_bytes, const void *wt, int64_t wt_bytes,
                     unsigned int *out, int ctas, void *stream);

/*
 * Diagnostic: the static-FP8 quantizer the kernels use, applied to n fp32
 * values y (device pointer): q[i] = e4m3_satfinite(y[i] / *scale), with
 * `scale` a device pointer to one fp32.  Values go through it in groups of
 * eight on the path the kernels take (paired arithmetic after the magnitude
 * clamp applied to bf16 y, or IEEE division for extreme scales).
 * Lets a test sweep every 16-bit y value against an independent encoder.
 */
int gnq_quantize_fp8_values(const float *y, int64_t n, const float *scale, uint8_t *q,
                            void *stream);

/*
 * Diagnostic: the element encoders the kernels use, applied to n fp32 values
 * v (device pointer): e4m3[i] = the E4M3 satfinite round-to-nearest-even code
 * of v[i], e2m1[i] = the E2M1 satfinite round-to-nearest-even code (low
 * nibble).  Either output may be NULL.  Lets a test compare the hardware
 * conversions with an independent encoder on special values (ties, zero
 * signs, subnormals, saturation).
 */
int gnq_encode_e4m3_e2m1(const float *v, int64_t n, uint8_t *e4m3,
                         uint8_t *e2m1, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GEMMA_NQ_H */
