/*
 * flce.h - C ABI of the fused linear cross-entropy library for GB300 (sm_103a).
 *
 * The operation (source: "Long-Sequence MoE RL Training: From First Principles
 * to MI300X", section 3 "Linear cross-entropy: don't build a 32 GB tensor to
 * get a scalar"): the language-model head forms logits Z = H W^T over
 * [tokens x vocab] and reduces every row through the softmax to a per-token
 * cross-entropy.  The fused method never stores Z: tokens are processed in
 * blocks, each block's logits are formed tile by tile and merged straight
 * into a per-row maximum and sum of exponentials, so a row keeps a handful of
 * scalars.  The backward forms the same logit tiles again, turns them into
 * dZ = softmax(Z) - onehot(target) (scaled by the upstream per-token gradient)
 * and contracts dZ into dH = dZ W and dW = dZ^T H, so no more than a
 * [block x vocab] slice of dZ exists at a time.
 * Section 2.3, Step 1 of "让长序列 MoE RL 训练更好调：Megatron-Lite / bumblebee
 * 的优化实践" describes the same loss as streaming along the vocab dimension.
 *
 * Notation: T tokens, Hd hidden size, V vocabulary size.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers of the current CUDA device and
 *     stay owned by the caller.  The library never allocates device memory:
 *     the caller passes a workspace of at least the size the matching
 *     *_workspace_size() function returns.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL means the legacy default stream).  Outputs are overwritten, never
 *     accumulated into.  Outputs must not overlap one another, the inputs or
 *     the workspace (not checked; overlapping buffers give undefined values).
 *     One workspace serves one call at a time: calls that share a workspace
 *     must be ordered on one stream.
 *   - Argument errors are detected on the host and returned before anything
 *     is launched.  Errors that depend on device data (a target outside
 *     [0, V) that is not ignore_index; a bounded wait inside a kernel that
 *     ran out) are written to a status word at the start of the workspace;
 *     read it with flce_read_device_status().  Each call clears that word
 *     first, so it reports the latest call made with this workspace.  Rows
 *     whose target is out of range are treated as ignored.
 *   - H and W are bf16, row-major: H [T, Hd], W [V, Hd], each row contiguous.
 *     Hd must be a positive multiple of 64; H, W, dH and dW must be 16-byte
 *     aligned; the workspace 256-byte aligned; every other array aligned to
 *     its element type (4 bytes for float, 8 for int64_t).  T may be 0.  V >= 1.
 *     T, V < 2^30.
 *   - Rows whose target equals ignore_index contribute zero loss and zero
 *     gradient and are not counted in n_valid.  ignore_index must lie outside
 *     [0, V).
 *   - Reductions: MEAN = sum over valid rows / n_valid (0 when n_valid == 0),
 *     SUM = sum over valid rows, NONE = one loss per token.
 *   - Results are deterministic: the same inputs and workspace size give
 *     bit-identical outputs on the same device.
 */
#ifndef FLCE_H_
#define FLCE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 1: the first interface.  2: the backward skips rows with a zero upstream
 * weight (its workspace holds the row list and the chunk's H rows),
 * flce_forward_valid, flce_score_valid and flce_backward_workspace_size_for_chunk
 * added, kernel kinds 6-8 added to the timing aid. */
#define FLCE_ABI_VERSION 2

#if defined(__GNUC__)
#define FLCE_API __attribute__((visibility("default")))
#else
#define FLCE_API
#endif

typedef enum flce_status {
  FLCE_OK = 0,
  FLCE_ERR_INVALID_ARG = 1,  /* null pointer, bad size, bad reduction, ignore_index in [0, V) */
  FLCE_ERR_UNSUPPORTED = 2,  /* Hd not a multiple of 64, or the device is not sm_103 */
  FLCE_ERR_ALIGNMENT = 3,    /* H, W, dH, dW not 16-byte aligned, the workspace not 256-byte, or a
                                per-token array not aligned to its element type */
  FLCE_ERR_WORKSPACE = 4,    /* workspace missing or smaller than required */
  FLCE_ERR_CUDA = 5,         /* a CUDA runtime / driver call failed; see flce_last_error() */
  FLCE_ERR_TARGET_RANGE = 6, /* device status: a target outside [0, V) and != ignore_index */
  FLCE_ERR_TIMEOUT = 7,      /* device status: a bounded wait inside a kernel ran out */
  FLCE_ERR_SEQUENCES = 8     /* device status: cu_seqlens decreases or leaves [0, T] */
} flce_status;

/* Element types of the tensors that may come in more than one. */
typedef enum flce_dtype { FLCE_DTYPE_BF16 = 0, FLCE_DTYPE_F32 = 1 } flce_dtype;

typedef enum flce_reduction {
  FLCE_REDUCTION_NONE = 0,
  FLCE_REDUCTION_MEAN = 1,
  FLCE_REDUCTION_SUM = 2,
  FLCE_REDUCTION_SEQUENCE_MEAN = 3 /* flce_policy_loss only */
} flce_reduction;

/* Bytes of workspace flce_forward() needs for these sizes (>= 256). */
FLCE_API size_t flce_forward_workspace_size(int64_t T, int64_t Hd, int64_t V);

/* Bytes of workspace flce_backward() needs to run with its default token
 * chunk.  The backward skips the rows whose upstream gradient g_t is zero
 * (ignored targets; their dZ rows vanish) and works on chunks of `chunk` of
 * the remaining rows, in token order; the workspace holds one [chunk x V] bf16
 * slice of dZ (the page's [block x vocab] residency), the chunk's rows of H
 * ([chunk x Hd] bf16) and O(T) scalars.  The default chunk is T rounded up to
 * 128 for T <= 256, else min(8192, T/2 rounded down to 128), so for T > 256 and
 * Hd < V/2 the workspace stays below the T*V*2 bytes of one dense bf16 logits
 * tensor.  A larger or smaller workspace is accepted:
 * the backward then uses the largest chunk (a multiple of 128 rows, at least
 * 128) that fits. */
FLCE_API size_t flce_backward_workspace_size(int64_t T, int64_t Hd, int64_t V);

/* Bytes of backward workspace for chunks of `chunk` rows (a positive multiple
 * of 128; chunks above T rounded up to 128 are capped there); 0 for an invalid
 * chunk or size. */
FLCE_API size_t flce_backward_workspace_size_for_chunk(int64_t T, int64_t Hd, int64_t V, int64_t chunk);

/* The token chunk flce_backward() uses with a workspace of `workspace_bytes`;
 * 0 if the workspace is too small. */
FLCE_API int64_t flce_backward_chunk_tokens(int64_t T, int64_t Hd, int64_t V, size_t workspace_bytes);

/* Forward.  Source: "Long-Sequence MoE RL Training: From First Principles to
 * MI300X", section 3 (logits H W^T reduced row-wise through the running-max /
 * log-sum-exp recurrence; loss per token).
 *   H        [T, Hd] bf16              hidden states
 *   W        [V, Hd] bf16              LM-head weight
 *   targets  [T] int64                 class per token, or ignore_index
 *   loss     [1] fp32 (MEAN, SUM) or [T] fp32 (NONE)
 *   lse      [T] fp32                  log sum_v exp(z_{t,v}) on every row
 *   logp     [T] fp32                  z_{t,y_t} - lse_t; 0 on ignored rows
 *   n_valid  [1] int64 or NULL         number of rows with a valid target
 *   workspace, workspace_bytes         >= flce_forward_workspace_size(T, Hd, V)
 * No [T x V] buffer exists at any time. */
FLCE_API flce_status flce_forward(const void* H, const void* W, const int64_t* targets, int64_t T, int64_t Hd,
                                  int64_t V, int64_t ignore_index, int32_t reduction, float* loss, float* lse,
                                  float* logp, int64_t* n_valid, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Forward for training: the same arguments and results as flce_forward(),
 * except that rows with an ignored target are left out of the contraction
 * altogether (their lse is written as 0; their loss and logp are 0 as always).
 * The rows with a valid target are listed in token order, their rows of H
 * gathered into the workspace, and the logit tiles run over that list only,
 * so masked tokens (padding, prompt prefixes) cost nothing but the copy; loss,
 * logp and the lse of listed rows are bit-identical to flce_forward()'s.  The
 * lse it returns is what flce_backward() needs (the backward reads it only on
 * rows with a non-zero upstream weight, which are valid rows).
 *   workspace, workspace_bytes  >= flce_forward_valid_workspace_size(T, Hd, V)
 *                               (the forward's, plus 8 bytes per token and the
 *                               [T x Hd] bf16 rows of H) */
FLCE_API size_t flce_forward_valid_workspace_size(int64_t T, int64_t Hd, int64_t V);
FLCE_API flce_status flce_forward_valid(const void* H, const void* W, const int64_t* targets, int64_t T, int64_t Hd,
                                        int64_t V, int64_t ignore_index, int32_t reduction, float* loss, float* lse,
                                        float* logp, int64_t* n_valid, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Backward.  Source: the same page and section (each logit tile is formed
 * again, turned into dZ = softmax - onehot and contracted into dH and dW
 * straight away).
 *   dloss    [1] fp32 (MEAN, SUM) or [T] fp32 (NONE): gradient of the loss output
 *   H, W, targets, T, Hd, V, ignore_index, reduction: as passed to flce_forward
 *   lse      [T] fp32                  the lse output of flce_forward (or flce_forward_valid)
 *                                      for these inputs
 *   dH       [T, Hd] bf16              overwritten with dL/dH (fp32 accumulation, rounded)
 *   dW       [V, Hd] fp32              overwritten with dL/dW, accumulated in fp32 over
 *                                      token chunks in a fixed order
 *   workspace, workspace_bytes         see flce_backward_workspace_size()
 * Per token, the upstream weight is g_t = dloss/n_valid (MEAN), dloss (SUM) or
 * dloss[t] (NONE), and 0 on ignored rows; dZ_{t,v} = g_t (exp(z_{t,v} - lse_t) - [v = y_t]). */
FLCE_API flce_status flce_backward(const float* dloss, const void* H, const void* W, const int64_t* targets,
                                   const float* lse, int64_t T, int64_t Hd, int64_t V, int64_t ignore_index,
                                   int32_t reduction, void* dH, float* dW, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Backward with a gradient on the logp output as well.  RL trainers build
 * their objective from the per-token log-probabilities (policy-gradient and
 * ratio terms), so the upstream gradient can arrive on logp instead of, or as
 * well as, on the loss.  On valid rows logp_t = -loss_t, so dlogp_t enters the
 * per-token weight as g_t = (gradient of the loss output at t) - dlogp_t.
 *   dloss   as flce_backward, or NULL (no gradient on the loss output)
 *   dlogp   [T] fp32, or NULL (no gradient on logp); ignored rows get g_t = 0
 * Everything else as flce_backward. */
FLCE_API flce_status flce_backward_logp(const float* dloss, const float* dlogp, const void* H, const void* W,
                                        const int64_t* targets, const float* lse, int64_t T, int64_t Hd, int64_t V,
                                        int64_t ignore_index, int32_t reduction, void* dH, float* dW,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* Forward without any allocation by the caller or the library.  The pages
 * have no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory at the point where they need the loss: code whose
 * framework allocator owns all of device memory, plugin hooks of inference or
 * training engines that are not allowed to allocate, and latency-critical
 * paths that forbid allocation.  Such callers pass only inputs and outputs.
 *
 * Arguments and results are those of flce_forward(); instead of a workspace,
 * the call uses a scratch array built into the library: a 32 MiB device array
 * that every GPU which loads the library holds until the process exits.  That
 * limits T to at most 253,952 tokens (any Hd and V); larger T is rejected with
 * FLCE_ERR_WORKSPACE before anything is launched.  The device status word of
 * the call (0, FLCE_ERR_TARGET_RANGE or FLCE_ERR_TIMEOUT) is copied into
 * *device_status (a device int32) unless it is NULL.
 *
 * The first call on a device looks up that device's address of the scratch
 * array (cudaGetSymbolAddress) with the device current; make that first call
 * before any stream capture.  All calls share the one array, and each call
 * overwrites what it needs from it, so calls whose kernels overlap on the GPU
 * (different streams, or different host threads on the same device) race and
 * give wrong results: order them on one stream. */
FLCE_API flce_status flce_forward_noalloc(const void* H, const void* W, const int64_t* targets, int64_t T,
                                          int64_t Hd, int64_t V, int64_t ignore_index, int32_t reduction,
                                          float* loss, float* lse, float* logp, int64_t* n_valid,
                                          int32_t* device_status, void* stream);

/* Scoring: per-token log p(target) and the greedy token, without a loss.
 * Serves comparing a trainer's token log-probabilities with a rollout
 * engine's (the token-level agreement checks of the pages' RL write-ups,
 * e.g. "Long-Sequence MoE RL Training: From First Principles to MI300X"
 * section 1: rollout then train).  Same logit tiles and log-sum-exp
 * recurrence as flce_forward; no reduction.
 *   logp    [T] fp32         z_{t,y_t} - lse_t; 0 on ignored rows
 *   lse     [T] fp32 or NULL
 *   argmax  [T] int64 or NULL  argmax_v z_{t,v} over the fp32-accumulated
 *                              logits, lowest id on ties
 *   workspace >= flce_score_workspace_size(T, Hd, V) */
FLCE_API size_t flce_score_workspace_size(int64_t T, int64_t Hd, int64_t V);
FLCE_API flce_status flce_score(const void* H, const void* W, const int64_t* targets, int64_t T, int64_t Hd, int64_t V,
                                int64_t ignore_index, float* logp, float* lse, int64_t* argmax, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Scoring over the rows with a valid target only: the same arguments and results
 * as flce_score(), except that rows with an ignored target are left out of the
 * contraction (lse 0, logp 0 and argmax -1 there); on every other row lse, logp
 * and argmax are bit-identical to flce_score()'s.  For scoring a rollout's
 * response tokens with the prompt masked.
 *   workspace, workspace_bytes  >= flce_score_valid_workspace_size(T, Hd, V) */
FLCE_API size_t flce_score_valid_workspace_size(int64_t T, int64_t Hd, int64_t V);
FLCE_API flce_status flce_score_valid(const void* H, const void* W, const int64_t* targets, int64_t T, int64_t Hd,
                                      int64_t V, int64_t ignore_index, float* logp, float* lse, int64_t* argmax,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* ---- vocab-parallel split ---------------------------------------------------
 * The vocabulary split into shards of consecutive rows, as when the LM head is
 * tensor-parallel over the vocab ("让长序列 MoE RL 训练更好调：Megatron-Lite /
 * bumblebee 的优化实践", section 2.3 Step 1: a 248,320-row vocab over two ranks
 * gives 124,160 columns per rank).  Each shard reduces its own logit columns to
 * a per-row log-sum-exp; the shards' partials combine exactly as the vocab
 * ranges inside one flce_forward call do (running max / log-sum-exp merge), so
 * the combined results equal flce_forward on the whole vocabulary.  Moving the
 * partials between ranks (an all-gather of 2 floats per token) and summing the
 * dH partials (an all-reduce) are the caller's collectives.
 *
 * Forward of one shard: W_shard [V_shard, Hd] holds global vocab rows
 * [vocab_offset, vocab_offset + V_shard) of a V_total vocabulary.
 *   shard_lse [T] fp32   log sum_{v in shard} exp(z_{t,v})
 *   shard_zy  [T] fp32   z_{t,y_t} when y_t lies in the shard, else 0
 *   workspace            >= flce_forward_workspace_size(T, Hd, V_shard)
 * ignore_index must lie outside [0, V_total). */
FLCE_API flce_status flce_forward_shard(const void* H, const void* W_shard, const int64_t* targets, int64_t T,
                                        int64_t Hd, int64_t V_shard, int64_t vocab_offset, int64_t V_total,
                                        int64_t ignore_index, float* shard_lse, float* shard_zy, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Bytes of workspace flce_combine_shards() needs (0 if n_shards is outside [1, 64]). */
FLCE_API size_t flce_combine_workspace_size(int64_t T, int32_t n_shards);

/* Combine the partials of n_shards shards (1..64), merged in shard order:
 *   shard_lse, shard_zy  [n_shards, T] fp32 (shard r's rows at offset r*T)
 * Outputs and reductions as flce_forward over the V_total vocabulary; targets
 * outside [0, V_total) that are not ignore_index set FLCE_ERR_TARGET_RANGE in
 * the workspace status word. */
FLCE_API flce_status flce_combine_shards(const float* shard_lse, const float* shard_zy, int32_t n_shards,
                                         const int64_t* targets, int64_t T, int64_t V_total, int64_t ignore_index,
                                         int32_t reduction, float* loss, float* lse, float* logp, int64_t* n_valid,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* Backward of one shard, given the combined lse [T]: dW_shard [V_shard, Hd]
 * fp32 is this shard's rows of dW; dH_partial [T, Hd] bf16 is this shard's
 * term sum_{v in shard} dZ_{t,v} w_v of dH (the shards' partials sum to dH).
 * g_t counts valid rows against the whole vocabulary.  Workspace as
 * flce_backward_workspace_size(T, Hd, V_shard). */
FLCE_API flce_status flce_backward_shard(const float* dloss, const void* H, const void* W_shard,
                                         const int64_t* targets, const float* lse, int64_t T, int64_t Hd,
                                         int64_t V_shard, int64_t vocab_offset, int64_t V_total, int64_t ignore_index,
                                         int32_t reduction, void* dH_partial, float* dW_shard, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* ---- the norm in front of the head ------------------------------------------
 * Residual add and root-mean-square norm, the last step before the LM head:
 *   h = x + residual, rounded to the residual's type (h = x without a residual)
 *   rstd_t = (mean_c h_{t,c}^2 + eps)^(-1/2),  y_{t,c} = h_{t,c} rstd_t w_c
 * over the rounded h, the value every later reader of the residual stream sees; the
 * squares are fp32, their sum and rstd carry what fp32 rounds off.  Any of three outputs:
 *   y        [T, Hd] bf16 or NULL   what flce_forward takes as H
 *   q        [T, Hd] e4m3 or NULL   y in 8 bits, what flce_linear_fp8 takes, with
 *   q_scale  [T, ceil(Hd/128)]      one E8M0 byte s per row and 128 channels: the value
 *                                   of an element is q 2^(s - 127).  2^(s - 127) is the
 *                                   smallest power of two, at least 2^-126, that brings
 *                                   the block's largest |y| to 448 or less; q is rounded
 *                                   once, from the product itself, to nearest even.  A
 *                                   NaN stays NaN and does not count for its block's
 *                                   scale; |h w| and h^2 have to stay within fp32.
 *   rstd     [T] fp32 or NULL       for the backward
 * Inputs: x [T, Hd] (row stride ldx elements), residual [T, Hd] (ldr) or NULL, each
 * bf16 or fp32 (flce_dtype), weight [Hd] bf16 or fp32.  h [T, Hd] (ldh, the
 * residual's type) is written when a residual is given and must be NULL
 * otherwise; it may be the residual itself (same pointer and stride) or, with
 * equal types, x itself.
 * Hd: a multiple of 16 up to 16384 (else FLCE_ERR_UNSUPPORTED).  Tensors 16-byte
 * aligned, row strides whole multiples of 16 bytes. */
FLCE_API flce_status flce_add_rms_norm(const void* x, int32_t x_dtype, int64_t ldx, const void* residual,
                                       int32_t residual_dtype, int64_t ldr, const void* weight, int32_t weight_dtype,
                                       int64_t T, int64_t Hd, float eps, void* h, int64_t ldh, void* y, float* rstd,
                                       void* q, uint8_t* q_scale, void* stream);

/* Its backward, for the gradient dy of y (bf16 or fp32) and, where h is read
 * elsewhere too, the gradient dh of h itself (h's type, or NULL):
 *   u = dy w,  dx = rstd (u - h rstd^2 mean_c(u h)) + dh,  dweight = sum_t dy h rstd
 *   dx       [T, Hd] h's type, contiguous   the gradient of x and of the residual alike
 *   dweight  [Hd] fp32                      summed in a fixed order
 * h and rstd as flce_add_rms_norm wrote them (h = x there without a residual).
 *   workspace, workspace_bytes  >= flce_add_rms_norm_backward_workspace_size(T, Hd) */
FLCE_API size_t flce_add_rms_norm_backward_workspace_size(int64_t T, int64_t Hd);
FLCE_API flce_status flce_add_rms_norm_backward(const void* dy, int32_t dy_dtype, int64_t lddy, const void* h,
                                                int32_t h_dtype, int64_t ldh, const void* weight,
                                                int32_t weight_dtype, const float* rstd, const void* dh, int64_t lddh,
                                                int64_t T, int64_t Hd, void* dx, float* dweight, void* workspace,
                                                size_t workspace_bytes, void* stream);

/* The norm for training with what its backward needs of h kept in 8 bits: the checkpoint takes
 * 1 + 1/128 bytes a channel instead of h's 2 or 4, and the backward reads as much.
 *   hq        [T, Hd] e4m3          h in 8 bits, rounded once, to nearest even
 *   hq_scale  [T, ceil(Hd/128)]     its E8M0 bytes, by q_scale's rule
 * h, y and rstd come from h itself and are bit-identical to flce_add_rms_norm's; y, rstd, hq and
 * hq_scale must all be given. */
FLCE_API flce_status flce_add_rms_norm_checkpoint(const void* x, int32_t x_dtype, int64_t ldx, const void* residual,
                                                  int32_t residual_dtype, int64_t ldr, const void* weight,
                                                  int32_t weight_dtype, int64_t T, int64_t Hd, float eps, void* h,
                                                  int64_t ldh, void* y, float* rstd, void* hq, uint8_t* hq_scale,
                                                  void* stream);

/* Its backward: flce_add_rms_norm_backward with h^ = hq 2^(hq_scale - 127) in the place of h
 * (rstd stays the forward's):
 *   u = dy w,  dx = rstd (u - h^ rstd^2 mean_c(u h^)) + dh,  dweight = sum_t dy h^ rstd
 * dh and dx have the type h_dtype.  An h^ is off by up to 2^-4 of h (and by 2^-10 of its scale);
 * dx and dweight are linear in such errors to first order and their mean is 0.
 *   workspace, workspace_bytes  >= flce_add_rms_norm_backward_workspace_size(T, Hd) */
FLCE_API flce_status flce_add_rms_norm_checkpoint_backward(const void* dy, int32_t dy_dtype, int64_t lddy,
                                                           const void* hq, const uint8_t* hq_scale, int32_t h_dtype,
                                                           const void* weight, int32_t weight_dtype, const float* rstd,
                                                           const void* dh, int64_t lddh, int64_t T, int64_t Hd, void* dx,
                                                           float* dweight, void* workspace, size_t workspace_bytes,
                                                           void* stream);

/* ---- the head's product in 8 bits ---------------------------------------------
 * For decoding (rollouts), and where logits are wanted as such (scores of given tokens
 * without [T x V] logits are flce_score's): logits from e4m3 operands with one
 * power-of-two scale (an E8M0 byte s, worth 2^(s - 127); 255 is NaN) per block of 128
 * along K.
 *
 * flce_quantize_fp8 lays out a matrix: a [rows, K] bf16 or fp32 (row stride lda)
 *   q        [rows, K] e4m3
 *   q_scale  [ceil(rows / block_rows), ceil(K/128)], block_rows 128 for weights (128 x 128
 *            blocks), 1 for activations; the scale rule is flce_add_rms_norm's, and an
 *            infinity saturates: +-448 at the scale of the largest finite numbers, 2^120. */
FLCE_API flce_status flce_quantize_fp8(const void* a, int32_t a_dtype, int64_t lda, int64_t rows, int64_t K,
                                       int32_t block_rows, void* q, uint8_t* q_scale, void* stream);

/* y[t, v] = sum_b 2^(x_scale[t, b] + W_scale[v / 128, b] - 254) sum_{k in block b} x[t, k] W[v, k]
 *   x [T, K] e4m3, x_scale [T, ceil(K/128)];  W [V, K] e4m3, W_scale [ceil(V/128), ceil(K/128)]
 *   y [T, V] bf16 or fp32 (y_dtype), row stride ldy >= V elements; nothing else is written
 * fp32 accumulation over the whole of K, one rounding to bf16.  K: a multiple of 16
 * (the last block may be short).  x and W 16-byte aligned and contiguous.
 *   workspace, workspace_bytes  >= flce_linear_fp8_workspace_size(T, K, V); its status word
 *                               reports FLCE_ERR_TIMEOUT */
FLCE_API size_t flce_linear_fp8_workspace_size(int64_t T, int64_t K, int64_t V);
FLCE_API flce_status flce_linear_fp8(const void* x, const uint8_t* x_scale, const void* W, const uint8_t* W_scale,
                                     int64_t T, int64_t K, int64_t V, void* y, int32_t y_dtype, int64_t ldy,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* ---- the head's product with 4-bit weights -------------------------------------
 * For decoding, which reading the weights bounds: as flce_linear_fp8, with half the bytes of
 * W.  The weights are e2m1 numbers (+-0, 0.5, 1, 1.5, 2, 3, 4, 6; two to a byte, the first of
 * two channels in its low bits) with one E8M0 scale per row and group of 32 channels.
 *
 * flce_quantize_fp4 lays out a matrix: a [rows, K] bf16 or fp32 (row stride lda), K a
 * multiple of 16, kb = ceil(K/128)
 *   q        [rows, 64 kb] bytes, filled up with zeros from channel K on; 16-byte aligned
 *            (flce_linear_fp4 wants 32)
 *   q_scale  [kb, rows, 4]: byte (b, r, j) is the scale of channels 128 b + 32 j .. + 31 of row r
 * Scale rule: the smallest 2^e with amax / 2^e <= 6, -126 <= e <= 125; numbers are rounded once,
 * to nearest even, and those above 6 2^125 saturate.  A group that holds a NaN gets the scale
 * NaN (255) and zeros. */
FLCE_API flce_status flce_quantize_fp4(const void* a, int32_t a_dtype, int64_t lda, int64_t rows, int64_t K, void* q,
                                       uint8_t* q_scale, void* stream);

/* y[t, v] = sum_g 2^(x_scale[t, g / 4] + W_scale[g / 4, v, g % 4] - 254) sum_{k in group g} x[t, k] W[v, k]
 *   x [T, K] e4m3, x_scale [T, kb] as flce_linear_fp8 takes them
 *   W [V, 64 kb] bytes, W_scale [kb, V, 4] as flce_quantize_fp4 writes them; numbers from channel K
 *   on must be zeros and their scales not NaN.  W 32-byte aligned, W_scale 4-byte aligned
 *   y, workspace as flce_linear_fp8's */
FLCE_API size_t flce_linear_fp4_workspace_size(int64_t T, int64_t K, int64_t V);
FLCE_API flce_status flce_linear_fp4(const void* x, const uint8_t* x_scale, const void* W, const uint8_t* W_scale,
                                     int64_t T, int64_t K, int64_t V, void* y, int32_t y_dtype, int64_t ldy,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* ---- drawing tokens ------------------------------------------------------------
 * One token for each row of logits, from a random number u in [0, 1) of its own, and the
 * logarithm of the probability it was drawn with (a rollout's old_logp).  With the row's logits
 * in descending order, equal ones by their index, and w_i = e^((l_i - max) / temperature):
 *   top-k  keeps the first k                                           (k <= 0: all)
 *   top-p  of those the shortest prefix whose w reach p times their sum (rounded to 53 bits),
 *          at least one                                                (p >= 1: all)
 *   min-p  those with w_i >= min_p w_max                               (min_p <= 0: all)
 * and the token is the first in vocabulary order whose cumulative kept w exceeds u times
 * the kept sum.  A temperature of 0 or less, or NaN, draws the largest logit of the lowest
 * index (logp 0).
 *   logits [T, V] bf16 or fp32, row stride ldl >= V elements, any alignment of their type.
 *          -inf and NaN are never drawn (a mask); where a row has +inf those alone are.  A row
 *          with nothing to draw gives the token ignore_index and logp 0.
 *   u      [T] fp32; below 0 and NaN count as 0, 1 and more as the number before 1
 *   temperature, top_k (int32), top_p, min_p: [T] of a setting for each row, or NULL: the
 *          number behind it for all (refused where negative or NaN, a temperature above 1e300
 *          (+inf), and top_p and min_p above 1; any top_k will do).  A row's temperature may be
 *          +inf: every w is then 1.  Temperatures below 1.44e-37 count as that
 *   tokens [T] int64;  logp [T] fp32 or NULL
 * Weights are rounded to whole multiples of a unit, the largest being 2^44 of them or more (2^46 up
 * to 131,071 words, 2^45 up to 262,143), and their sums are exact, so the result does not depend on
 * the order of summation.  V up to 393,216.  ignore_index lies outside [0, V). */
FLCE_API flce_status flce_sample(const void* logits, int32_t dtype, int64_t ldl, const float* u, int64_t T, int64_t V,
                                 const float* temperature, double temperature_all, const int32_t* top_k,
                                 int64_t top_k_all, const float* top_p, double top_p_all, const float* min_p,
                                 double min_p_all, int64_t ignore_index, int64_t* tokens, float* logp, void* stream);

/* ---- objectives on logp ------------------------------------------------------
 * Both take the per-token log-probabilities that the forward returns and give
 * the gradient that flce_backward_logp takes as dlogp: forward, loss, backward
 * without a host step in between.  Tokens whose target is ignore_index do not
 * count: whatever logp, old_logp, ref_logp or the advantages hold there (NaN
 * and infinities included) has no effect, and their dlogp is 0.
 *
 * cu_seqlens [n + 1] int64 gives the packed sequences: sequence i is the tokens
 * cu_seqlens[i] .. cu_seqlens[i + 1] - 1; empty ones are allowed, and a token in no
 * sequence (before cu_seqlens[0], from cu_seqlens[n] on) is treated as ignored.  If it
 * decreases or leaves [0, T] the device status is FLCE_ERR_SEQUENCES and the
 * outputs mean nothing (no access leaves the arrays).
 *
 * Either of loss and dlogp may be NULL.  dloss is the gradient of the loss
 * output ([1], or one per loss entry with NONE), NULL for ones. */

/* Clipped policy loss with a KL term.  Per valid token, with
 *   d = logp - old_logp clamped to [-20, 20],  rho = e^d,  A the advantage:
 *   pg = -min(rho A, clip(rho, 1 - clip_low, 1 + clip_high) A)
 *        and, with dual_clip c > 1 and A < 0, at most -c A (dual_clip 0: no such limit)
 *   e = ref_logp - logp;  kl = -e (K1), e^2 / 2 (K2), e^e - 1 - e (K3, e clamped like d)
 *   L = pg + kl_coef kl
 * loss = sum over valid tokens / n_valid (MEAN), the sum (SUM), one per token (NONE),
 * or (SEQUENCE_MEAN) the mean over the sequences that have a valid token of each
 * one's mean.  The gradient of pg is -A rho where rho is not clipped and d not
 * clamped, else 0.  No valid token: loss and stats are 0.
 *   logp, old_logp [T] fp32; ref_logp [T] fp32 or NULL (kl = 0; kl_coef must be 0)
 *   advantages [T] fp32, or [n_seqs] with advantages_per_sequence
 *   cu_seqlens [n_seqs + 1] or NULL (one stretch of T tokens); needed by
 *              SEQUENCE_MEAN and advantages_per_sequence
 *   dlogp   [T] fp32
 *   stats   [4] fp32 or NULL: means over the valid tokens of kl, of "clipped"
 *           (either way), of d and of rho
 *   n_valid [1] int64 or NULL
 *   workspace >= flce_policy_loss_workspace_size(T, n_seqs) */
typedef enum flce_kl { FLCE_KL_K1 = 1, FLCE_KL_K2 = 2, FLCE_KL_K3 = 3 } flce_kl;
FLCE_API size_t flce_policy_loss_workspace_size(int64_t T, int64_t n_seqs);
FLCE_API flce_status flce_policy_loss(const float* dloss, const float* logp, const float* old_logp,
                                      const float* ref_logp, const float* advantages,
                                      int32_t advantages_per_sequence, const int64_t* targets,
                                      const int64_t* cu_seqlens, int64_t n_seqs, int64_t T, int64_t ignore_index,
                                      int32_t reduction, float clip_low, float clip_high, float dual_clip,
                                      float kl_coef, int32_t kl_kind, float* loss, float* dlogp, float* stats,
                                      int64_t* n_valid, void* workspace, size_t workspace_bytes, void* stream);

/* Preference loss on paired log ratios.  Sequence 2p is pair p's chosen answer,
 * 2p + 1 the rejected one.  S_i = sum over sequence i's valid tokens of
 * logp - ref_logp (of logp without ref_logp), divided by their number with
 * length_normalize; 0 for a sequence without one.  D_p = S_{2p} - S_{2p+1},
 * h = beta D - margin:
 *   SIGMOID  (1 - label_smoothing) softplus(-h) + label_smoothing softplus(h)
 *   HINGE    max(0, 1 - h)
 *   IPO      (D - 1 / (2 beta))^2
 * loss = the mean over all n_pairs pairs, the sum, or one per pair (NONE).
 *   cu_seqlens [2 n_pairs + 1]
 *   chosen_rewards, rejected_rewards [n_pairs] fp32 or NULL: beta S
 *   workspace >= flce_preference_loss_workspace_size(n_pairs) */
typedef enum flce_preference {
  FLCE_PREFERENCE_SIGMOID = 0,
  FLCE_PREFERENCE_HINGE = 1,
  FLCE_PREFERENCE_IPO = 2
} flce_preference;
FLCE_API size_t flce_preference_loss_workspace_size(int64_t n_pairs);
FLCE_API flce_status flce_preference_loss(const float* dloss, const float* logp, const float* ref_logp,
                                          const int64_t* targets, const int64_t* cu_seqlens, int64_t n_pairs,
                                          int64_t T, int64_t ignore_index, int32_t reduction, int32_t kind, float beta,
                                          float label_smoothing, float margin, int32_t length_normalize, float* loss,
                                          float* dlogp, float* chosen_rewards, float* rejected_rewards,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* Synchronizes `stream`, then reads the device status word of the latest call
 * made with `workspace` into *out (an flce_status value). */
FLCE_API flce_status flce_read_device_status(const void* workspace, void* stream, int32_t* out);

/* Self-test of the kernels' bounded waits (no counterpart on the pages): one
 * thread waits on an mbarrier that nothing ever completes, with the same
 * bounded wait every GEMM role uses, and writes FLCE_ERR_TIMEOUT to the status
 * word of `workspace` (>= 256 bytes) once `timeout_ns` (1e6 .. 1e10) has
 * passed.  Read it with flce_read_device_status(); the context stays usable. */
FLCE_API flce_status flce_selftest_wait_timeout(void* workspace, uint64_t timeout_ns, void* stream);

/* Human-readable name of a status code (static storage). */
FLCE_API const char* flce_status_string(int32_t status);

/* Text of the last FLCE_ERR_CUDA / argument error raised on this host thread. */
FLCE_API const char* flce_last_error(void);

/* FLCE_ABI_VERSION of the loaded library. */
FLCE_API int32_t flce_abi_version(void);

/* Limit, in nanoseconds, of every bounded wait inside the kernels.  Values
 * below 1e6 are raised to 1e6.  Affects later launches only.  Until this is
 * called the limit of each launch is max(4e9, 16 x K) ns, K being the longest
 * contraction of one output tile in that launch (Hd in the forward and dZ
 * kernels; V for dH tiles and the token chunk for dW tiles), since the longest
 * wait spans one tile's K loop (about 8 SM-pair clocks per unit of K); once it
 * is called, the given value is used for every launch. */
FLCE_API void flce_set_wait_timeout_ns(uint64_t ns);

/* ---- per-kernel timing, a profiling aid ------------------------------------
 * While enabled, every kernel launch of the library is bracketed by CUDA
 * events recorded on its launch stream.  flce_profile_collect() synchronizes
 * on those events and returns, per kernel kind, the launches, the summed
 * device time and the summed algorithmic work (FLOPs and bytes the kernel's
 * mathematics requires, independent of how it is executed).  The backward's
 * work is counted over the rows it does not skip; that count is read from the
 * backward workspace at collection time, so collect while the workspaces of
 * the profiled calls still exist (each reports its latest call). */
typedef struct flce_kernel_stats {
  int32_t kind;     /* flce_kernel_kind value */
  int32_t launches;
  double total_ms;
  double flops;     /* algorithmic FLOPs summed over the launches */
  double bytes;     /* algorithmic DRAM bytes summed over the launches */
} flce_kernel_stats;

typedef enum flce_kernel_kind {
  FLCE_KERNEL_FWD_LOGITS_LSE = 0, /* logit tiles H W^T + running max / sum-exp epilogue */
  FLCE_KERNEL_FWD_FINALIZE = 1,   /* per-row lse / loss / logp and block partial sums */
  FLCE_KERNEL_FWD_REDUCE = 2,     /* fixed-order scalar loss and n_valid */
  FLCE_KERNEL_BWD_PREP = 3,       /* n_valid and the per-token upstream weights g */
  FLCE_KERNEL_BWD_DZ = 4,         /* recomputed logit tiles + dZ epilogue, bf16 dZ chunk */
  FLCE_KERNEL_BWD_DH_DW = 5,      /* dH chunk = dZ W and dW (+)= dZ^T H, one launch per chunk */
  FLCE_KERNEL_BWD_GATHER = 6,     /* the chunk's rows of H gathered through the row list */
  FLCE_KERNEL_BWD_SCATTER = 7,    /* not launched: the dH tiles write their rows straight to their tokens */
  FLCE_KERNEL_FWD_LIST = 8,       /* flce_forward_valid: the list of rows with a valid target */
  FLCE_KERNEL_ADD_RMS_NORM = 9,   /* residual add, norm, 8-bit output */
  FLCE_KERNEL_NORM_BWD = 10,      /* dx and each block's share of dweight */
  FLCE_KERNEL_NORM_DW = 11,       /* the shares' fixed-order sum */
  FLCE_KERNEL_POLICY_LOSS = 12,   /* flce_policy_loss, all launches of a call */
  FLCE_KERNEL_PREFERENCE_LOSS = 13, /* flce_preference_loss, all launches of a call */
  FLCE_KERNEL_QUANTIZE_FP8 = 14,  /* a matrix to e4m3 with block scales */
  FLCE_KERNEL_LINEAR_FP8 = 15,    /* the 8-bit head product */
  FLCE_KERNEL_QUANTIZE_FP4 = 16,  /* a matrix to e2m1 with group scales */
  FLCE_KERNEL_LINEAR_FP4 = 17,    /* the head product with 4-bit weights */
  FLCE_KERNEL_SAMPLE = 18,        /* tokens drawn from logits */
  FLCE_KERNEL_KINDS = 19
} flce_kernel_kind;

FLCE_API void flce_profile_enable(int32_t on);
/* Fills up to `max_entries` records (one per kind that launched), sets *n_out,
 * and clears the records.  Returns FLCE_ERR_CUDA if an event query fails. */
FLCE_API flce_status flce_profile_collect(flce_kernel_stats* out, int32_t max_entries, int32_t* n_out);
FLCE_API const char* flce_kernel_name(int32_t kind);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_H_ */
