/*
 * zero.h -- C ABI of libzero: the ZeRO sharded update on one MI355X (gfx950).
 *
 * N data-parallel ranks are simulated as N buffers in one GPU's HBM.  The
 * library reduces the ranks' BF16 gradient contributions element-wise in FP32
 * and hands each owner its 1/N slice (reduce-scatter), applies the owner's
 * fused mixed-precision Adam/AdamW update to its FP32 master, m and v shards
 * and writes its BF16 working-weight shard, gathers BF16 shards into a
 * temporary full per-layer view (all-gather), and streams a gradient shard
 * that lives in pinned host memory through two device slots (offload).
 *
 * The method is described on three web pages, cited below by title and
 * section:
 *   [slide] "分担数据，与分担保存责任，是两个动作" (beats b0-b3, notes 原 N46-N48)
 *   [essay] "把训练账本放进多张设备" (sections 从持久状态开始记账,
 *           数据分工与保存分工, ZeRO-3 的一次完整计算)
 *   [blog]  "数据并行与 ZeRO：三级分片各省多少" (sections 每个参数 16 字节,
 *           三级分片, 分片放到 CPU：两个缓冲就够)
 *
 * Conventions shared by every call:
 *  - Device buffers are plain device pointers; the library never allocates,
 *    frees or takes ownership of any caller buffer.  Host arrays (pointer
 *    tables, weights, counts, hyper-parameters) are read during the call only.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Every
 *    compute call is asynchronous on that stream and does not synchronise.
 *  - Each call validates all its arguments before launching anything; on a
 *    validation failure nothing is launched and nothing is written.
 *  - Return value: ZERO_OK (0) or a negative zero_status.  zero_last_error()
 *    gives a message for the last failure on the calling thread.
 *  - Element counts of 0 are valid and launch nothing; the buffer pointers of
 *    such a call are not used and may be NULL (the pointer tables may not).
 *  - Input and output buffers must not overlap, except where a call says so.
 *  - Floating point: binary32 arithmetic with one rounding per operation (no
 *    contraction into FMA), correctly rounded division and square root, FP32
 *    subnormals preserved; BF16 values are rounded to nearest-even.  Results
 *    are therefore the same bits on every call with the same inputs.
 *  - Calls on different streams are independent; an offload handle must not be
 *    used from two threads at once.
 */
#ifndef ZERO_H
#define ZERO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_MAX_RANKS 16   /* upper bound on n_ranks and n_shards */
#define ZERO_NORM_BLOCKS 1024  /* partial sums per shard in zero_grad_norm_sq */
#define ZERO_OFFLOAD_MAX_CHUNKS 65536  /* upper bound on ceil(shard/chunk) of an offload handle */
/* doubles in the library's own partial-sum array of zero_grad_norm_sq_no_alloc (128 KiB per GPU) */
#define ZERO_NORM_SCRATCH_DOUBLES (ZERO_MAX_RANKS * ZERO_NORM_BLOCKS)

/* limits of zero_newton_schulz */
#define ZERO_NS_MAX_STEPS 16
#define ZERO_NS_MAX_MATS 65535
#define ZERO_NS_MAX_SIDE 262144
#define ZERO_NS_MAX_SIGMA 2   /* largest singular value a step may give */
#define ZERO_NS_MAX_GAIN 16   /* largest |p(s)/s| of a step */

/* 8-bit activations and the feed-forward block */
#define ZERO_ACT8_BLOCK 32   /* neighbours of a row that share a power of two */
#define ZERO_ACT8_MAX_COLS 2147483648
#define ZERO_ACT8_MAX_VALUES 34359738368   /* rows filled up to whole blocks */
#define ZERO_FFN_MAX_TOKENS 16777216
#define ZERO_FFN_MAX_SIDE 262144
#define ZERO_FFN_MAX_STRIDE 8388608
#define ZERO_FFN_BACKWARD 1    /* flags of zero_ffn_workspace */
#define ZERO_FFN_UNALIGNED 2

typedef enum zero_status {
  ZERO_OK = 0,
  ZERO_ERR_ARG = -1,    /* null pointer, count out of range, overlapping buffers, bad hyper-parameter */
  ZERO_ERR_ALIGN = -2,  /* a pointer is not aligned to its element size */
  ZERO_ERR_SIZE = -3,   /* sizes inconsistent with each other */
  ZERO_ERR_HIP = -4,    /* the HIP runtime reported an error (see zero_last_error) */
  ZERO_ERR_STATE = -5   /* an offload handle was used out of order */
} zero_status;

/* Adam / AdamW hyper-parameters of one update.  step is t >= 1. */
typedef struct zero_adam_hparams {
  float lr, beta1, beta2, eps, weight_decay;
  int64_t step;
} zero_adam_hparams;

/* The per-step scalars the update kernel uses, all binary32:
 * one_minus_beta_i = 1 - beta_i (a float32 subtraction),
 * bias_correction_i = float32(1 - double(beta_i)^step). */
typedef struct zero_adam_scalars {
  float lr, beta1, beta2, one_minus_beta1, one_minus_beta2;
  float bias_correction1, bias_correction2, eps, weight_decay;
} zero_adam_scalars;

/* ---------------------------------------------------------------- host-side metadata */

/* Fill `out` with the scalars that zero_adam_shard_step uses for `hp`.
 * Errors: ZERO_ERR_ARG if a pointer is NULL, hp->step < 1, or a beta is not
 * in [0, 1). */
int zero_adam_scalars_compute(const zero_adam_hparams* hp, zero_adam_scalars* out);

/* Loss-normalisation weights of the reduction ([slide] note 原 N48: scale the
 * reduction to match the objective; [essay] 数据分工与保存分工: ranks with
 * different sample or token counts must not be weighted blindly alike).
 * counts == NULL: w_r = 1/n_ranks (batch mean).  Otherwise
 * w_r = float32(double(counts[r]) / double(sum counts)).
 * weights_out: host array of n_ranks floats.
 * Errors: ZERO_ERR_ARG for NULL weights_out, n_ranks outside [1, 16], a
 * negative count or a zero sum. */
int zero_rank_weights(const int64_t* counts, int n_ranks, float* weights_out);

/* Flatten/pad/partition layout of one unit ([slide] note 原 N46: owner shards
 * are slices of the parameters, not layers; [blog] 三级分片: each owner holds
 * 1/N).  psi = sum of numels; psi_pad = psi rounded up to a multiple of
 * n_shards*256; shard_numel = psi_pad / n_shards.  Shard k of the flat vector
 * is [k*shard_numel, (k+1)*shard_numel).
 * Errors: ZERO_ERR_ARG for NULL outputs, numels == NULL with n_tensors > 0,
 * n_shards outside [1, 16] or a negative numel; ZERO_ERR_SIZE on overflow. */
int zero_shard_layout(const int64_t* numels, int n_tensors, int n_shards,
                      int64_t* psi, int64_t* psi_pad, int64_t* shard_numel);

/* ---------------------------------------------------------------- device calls */

/* Reduce-scatter ([slide] note 原 N48; [essay] ZeRO-3 的一次完整计算;
 * [blog] 三级分片, ZeRO-2): the contributions of every rank to the SAME
 * parameter are combined element-wise, and owner k receives only its slice.
 *
 *   rank_grads   host array of n_ranks device pointers; rank r's contribution
 *                is `numel` BF16 values (bit patterns) at rank_grads[r].
 *   rank_weights host array of n_ranks floats (see zero_rank_weights).
 *   shards_out   host array of n_shards device pointers to FP32 buffers of
 *                numel/n_shards elements each.
 *   accumulate   0: out = red;  1: out = out + red   (in place).
 *
 * For element i of shard k (global index j = k*numel/n_shards + i):
 *   red = w_0*x_0[j];  red = red + w_r*x_r[j] for r = 1..n_ranks-1,
 * with x_r the exact FP32 widening of the BF16 value: a fixed rank order, so
 * the result is bitwise reproducible.  n_shards = 1 with pre-sliced
 * contributions is the owner-local form (buckets, offload chunks).
 * Errors: ZERO_ERR_ARG (NULL pointers, n_ranks or n_shards outside [1, 16],
 * numel < 0, buffers overlapping), ZERO_ERR_SIZE (numel % n_shards != 0),
 * ZERO_ERR_ALIGN (a BF16 pointer not 2-byte or FP32 pointer not 4-byte
 * aligned), ZERO_ERR_HIP (launch failure). */
int zero_reduce_scatter(const uint16_t* const* rank_grads, const float* rank_weights, int n_ranks,
                        int64_t numel, float* const* shards_out, int n_shards, int accumulate,
                        void* stream);

/* zero_reduce_scatter for FP32 contributions (gradients kept in FP32: the
 * +2 bytes per parameter variant of [blog] 每个参数 16 字节).  Same
 * arithmetic and order; rank_grads[r] points to numel FP32 values (4-byte
 * aligned).  The vector path needs 16-byte aligned pointers and
 * numel/n_shards % 4 == 0. */
int zero_reduce_scatter_f32(const float* const* rank_grads, const float* rank_weights, int n_ranks,
                            int64_t numel, float* const* shards_out, int n_shards, int accumulate,
                            void* stream);

/* Owner update: one fused pass of mixed-precision Adam/AdamW over n elements
 * of the owner's shard ([slide] note 原 N48: the owner updates its master
 * weights and m/v with the combined gradient; [essay] 从持久状态开始记账 and
 * [blog] 每个参数 16 字节: FP32 master, two FP32 moments, BF16 working weight).
 *
 *   master, exp_avg, exp_avg_sq  FP32[n] device, updated in place.
 *   bf16_out                     BF16[n] device, written: the new working weights.
 *   grad                         FP32[n] device, read (the reduced gradient shard).
 *
 * Per element, with the scalars of zero_adam_scalars_compute:
 *   m' = b1*m + (1-b1)*g;  v' = b2*v + (1-b2)*(g*g);
 *   u = (m'/bc1) / (sqrt(v'/bc2) + eps);  if wd != 0: u = u + wd*p;
 *   p' = p - lr*u;  bf16_out = round_to_nearest_even_bf16(p').
 * Non-finite values propagate by IEEE rules (no clipping or skipping).
 * Errors: ZERO_ERR_ARG (NULL, n < 0, overlap, bad hyper-parameters),
 * ZERO_ERR_ALIGN, ZERO_ERR_HIP. */
int zero_adam_shard_step(float* master, float* exp_avg, float* exp_avg_sq, uint16_t* bf16_out,
                         const float* grad, int64_t n, const zero_adam_hparams* hp, void* stream);

/* zero_adam_shard_step with the gradient first multiplied by a device scalar:
 * g = g * (*grad_scale) (one binary32 multiply), then the same update.  Used
 * with the clip coefficient of zero_grad_norm_sq, which stays on the device.
 *   grad_scale   device pointer to one float (4-byte aligned), read once; it
 *                may not lie inside master, exp_avg, exp_avg_sq or bf16_out.
 * Errors: as zero_adam_shard_step; ZERO_ERR_ARG for a NULL grad_scale or one
 * inside a buffer the update writes. */
int zero_adam_shard_step_scaled(float* master, float* exp_avg, float* exp_avg_sq,
                                uint16_t* bf16_out, const float* grad, const float* grad_scale,
                                int64_t n, const zero_adam_hparams* hp, void* stream);

/* Global gradient norm and clip coefficient (optional; the pages do not
 * describe clipping).  norm_sq_out[0] = sum over the shards of x*x, each square
 * exact in FP64 and the additions in FP64 in an order fixed by shard_numel and
 * n_shards alone (per shard ZERO_NORM_BLOCKS or fewer lane-sequential partial
 * sums, a butterfly over each 64-lane wave, the 4 waves of a block in order,
 * then the per-block partial sums in index order), so repeated calls give the
 * same bits on any device.  If clip_coef_out is not NULL it receives
 * float(min(1, max_norm / (sqrt(norm_sq) + 1e-6))) computed in FP64.
 *   shards       host array of n_shards device pointers to FP32[shard_numel].
 *   workspace    device scratch of workspace_len >= n_shards*ZERO_NORM_BLOCKS
 *                doubles (8-byte aligned), overwritten.
 *   norm_sq_out  device pointer to one double.
 * Errors: ZERO_ERR_ARG (NULL, counts, overlap, max_norm <= 0 with a clip
 * output), ZERO_ERR_SIZE (workspace too small), ZERO_ERR_ALIGN, ZERO_ERR_HIP. */
int zero_grad_norm_sq(const float* const* shards, int n_shards, int64_t shard_numel,
                      double* workspace, int64_t workspace_len, double* norm_sq_out,
                      float max_norm, float* clip_coef_out, void* stream);

/* zero_grad_norm_sq without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  The per-block partial sums go to an array
 * of ZERO_NORM_SCRATCH_DOUBLES doubles (128 KiB) that the library itself
 * holds in every GPU it runs on, until the process ends; its address on a
 * device is looked up on the first call with that device current.  The call
 * allocates nothing (no hipMalloc, hipFree or allocating library routine).
 * Same kernels, summation order and bits as zero_grad_norm_sq.
 *   shards, n_shards, shard_numel, norm_sq_out, max_norm, clip_coef_out,
 *   stream: as zero_grad_norm_sq.
 * Every call on one GPU uses that GPU's one array: calls that overlap in time
 * on one GPU (other streams, other threads) race on it and give wrong
 * results, so the caller serialises them.  Nothing carries over between
 * calls: each call's first pass writes every partial sum its second pass
 * reads, so the array needs no clearing.
 * Errors: as zero_grad_norm_sq; ZERO_ERR_SIZE if n_shards*ZERO_NORM_BLOCKS
 * partial sums would not fit the array (not reachable with n_shards <= 16);
 * ZERO_ERR_HIP if the array's device address cannot be obtained. */
int zero_grad_norm_sq_no_alloc(const float* const* shards, int n_shards, int64_t shard_numel,
                               double* norm_sq_out, float max_norm, float* clip_coef_out,
                               void* stream);

/* Reduce-scatter and owner update in one pass ([blog] 三级分片, ZeRO-1: the
 * optimizer step sits between the reduce-scatter and the all-gather).  For
 * every owner k it computes exactly zero_reduce_scatter's shard k (without
 * storing it unless grad_out is given) and applies zero_adam_shard_step's
 * update to owner k's state with it, so the results are bit-identical to the
 * two calls in sequence, with 8 fewer bytes of HBM traffic per parameter.
 *
 *   rank_grads, rank_weights, n_ranks, numel, n_shards: as zero_reduce_scatter.
 *   master, exp_avg, exp_avg_sq  host arrays of n_shards device pointers to
 *                FP32 state of numel/n_shards elements each (updated in place).
 *   bf16_out     host array of n_shards device pointers to BF16 working shards.
 *   grad_acc     NULL, or a host array of n_shards device pointers to FP32
 *                accumulated gradients: the update then uses grad_acc[k] + red,
 *                exactly zero_reduce_scatter's accumulate mode (the last
 *                micro-batch of an accumulation, updating directly).
 *   grad_out     NULL, or a host array of n_shards device pointers to FP32
 *                buffers that receive the (accumulated) reduced shards;
 *                grad_out[k] may equal grad_acc[k] (in place).
 * Errors: as zero_reduce_scatter and zero_adam_shard_step; every output must
 * be disjoint from every other buffer except grad_out[k] == grad_acc[k]. */
int zero_reduce_scatter_adam(const uint16_t* const* rank_grads, const float* rank_weights,
                             int n_ranks, int64_t numel, int n_shards, float* const* master,
                             float* const* exp_avg, float* const* exp_avg_sq,
                             uint16_t* const* bf16_out, const float* const* grad_acc,
                             float* const* grad_out, const zero_adam_hparams* hp, void* stream);

/* Graph-capturable forms of the owner update and of the fused call: the same
 * operations ([slide] note 原 N48: the owner updates its master weights and
 * m/v with the combined gradient; [blog] 三级分片, ZeRO-1: the step between
 * the reduce-scatter and the all-gather) and the same arithmetic, with the
 * step's scalars read from device memory when the kernel runs instead of
 * being passed by value at the call.  A caller that captures a step into a
 * HIP graph puts each step's scalars (zero_adam_scalars_compute on the host)
 * into the device struct before the update kernels of each replay run: with a
 * copy on the replay stream, or with zero_adam_scalars_fetch captured as the
 * graph's first kernel; the captured launches then apply that step's bias
 * corrections.
 * The decay term is applied when the device struct's weight_decay is non-zero,
 * exactly as the host-scalar forms decide it, so results are bit-identical to
 * zero_adam_shard_step / zero_adam_shard_step_scaled / zero_reduce_scatter_adam
 * with the hyper-parameters the scalars were computed from.  Rank weights are
 * still passed by value (a captured graph keeps the weights of the capture).
 *
 *   scalars_dev  device pointer to one zero_adam_scalars (4-byte aligned),
 *                filled by the caller from zero_adam_scalars_compute; it may
 *                not overlap a buffer the call writes.  Its values are not
 *                validated (they were, when computed).
 *   grad_scale   (zero_adam_shard_step_dev) NULL, or a device float the
 *                gradient is multiplied by, as in zero_adam_shard_step_scaled.
 * Errors: as the host-scalar forms, without the hyper-parameter checks, plus
 * ZERO_ERR_ARG / ZERO_ERR_ALIGN for scalars_dev. */
int zero_adam_shard_step_dev(float* master, float* exp_avg, float* exp_avg_sq, uint16_t* bf16_out,
                             const float* grad, const float* grad_scale, int64_t n,
                             const zero_adam_scalars* scalars_dev, void* stream);
int zero_reduce_scatter_adam_dev(const uint16_t* const* rank_grads, const float* rank_weights,
                                 int n_ranks, int64_t numel, int n_shards, float* const* master,
                                 float* const* exp_avg, float* const* exp_avg_sq,
                                 uint16_t* const* bf16_out, const float* const* grad_acc,
                                 float* const* grad_out, const zero_adam_scalars* scalars_dev,
                                 void* stream);

/* Scalar staging for captured steps, as a kernel instead of a copy: one
 * single-lane kernel on `stream` copies slot (*cursor_dev mod ring_len) of a
 * ring of zero_adam_scalars in pinned host memory into scalars_dev, then adds
 * one to *cursor_dev.  A step captured into a HIP graph starts with this call
 * (then the _dev calls read scalars_dev), so each replay takes the next slot
 * with no host-to-device copy between replays.  Protocol: *cursor_dev is 0
 * before the first replay (cleared by the caller before capture); the host
 * writes step t's scalars (zero_adam_scalars_compute) into slot t mod
 * ring_len before launching replay t, and rewrites a slot only after the
 * replay that read it has completed.  The ring is read with system-scope
 * loads when the kernel runs, so host writes made before the launch are seen.
 *
 *   ring_host    ring_len consecutive zero_adam_scalars in memory from
 *                hipHostMalloc (pinned, mapped for the device), 4-byte aligned
 *   ring_len     a power of two, 1..65536 (so that the slot sequence stays
 *                the same when the 32-bit cursor wraps)
 *   cursor_dev   device uint32_t, 4-byte aligned, read and written
 *   scalars_dev  device zero_adam_scalars, 4-byte aligned, written
 * Ownership: all four buffers belong to the caller.
 * Errors: ZERO_ERR_ARG for NULL pointers, ring_len out of range, cursor and
 * scalars overlapping, or a ring that is not one pinned host allocation
 * holding ring_len structs (checked with the runtime's pointer attributes);
 * ZERO_ERR_ALIGN for misaligned pointers.  Nothing is launched on error. */
int zero_adam_scalars_fetch(const zero_adam_scalars* ring_host, int ring_len, uint32_t* cursor_dev,
                            zero_adam_scalars* scalars_dev, void* stream);

/* All-gather into a temporary full view ([slide] note 原 N47 and beat b2;
 * [essay] ZeRO-3 的一次完整计算; [blog] 三级分片, ZeRO-3): the owners'
 * shards, concatenated in owner order, form the full per-layer view.
 *
 *   shards       host array of n_shards device pointers, shard_bytes each.
 *   full_view    device buffer of n_shards*shard_bytes bytes, written; owned
 *                by the caller, who releases it after use.
 * A byte copy, so it serves any element type.  Errors: ZERO_ERR_ARG (NULL,
 * n_shards outside [1, 16], shard_bytes < 0, overlap), ZERO_ERR_HIP. */
int zero_all_gather_layer(const void* const* shards, int n_shards, int64_t shard_bytes,
                          void* full_view, void* stream);

/* ---------------------------------------------------------------- Muon step
 *
 * The optimizer whose only state is the first moment ([blog] 每个参数 16 字节
 * counts its 12 bytes per parameter: BF16 weight and gradient, FP32 master and
 * momentum): the momentum of every weight matrix is orthogonalised by
 * Newton-Schulz products before it is applied.  Its step over sharded units:
 *   1. zero_reduce_scatter_muon (or zero_reduce_scatter, a gradient norm and
 *      zero_muon_momentum): every owner's momentum shard and the BF16
 *      directions of its slice;
 *   2. zero_all_gather_layer of the directions: the orthogonalisation needs
 *      whole matrices;
 *   3. zero_newton_schulz on each stack of equal matrices in the view;
 *   4. zero_muon_shard_step on each owner's slice of the result;
 *   5. zero_all_gather_layer of the working weights, as after any update. */
typedef struct zero_muon_hparams {
  float lr;            /* learning rate */
  float momentum;      /* b, in [0, 1) */
  float weight_decay;  /* decoupled, scaled by lr */
  int32_t nesterov;    /* 1: look-ahead direction; 0: the momentum itself */
} zero_muon_hparams;

/* zero_newton_schulz's input types */
enum { ZERO_BF16 = 0, ZERO_FP32 = 1 };

/* Momentum step over n elements of an owner's shard.
 *   momentum       FP32[n] device, updated in place.
 *   direction_out  BF16[n] device, written.
 *   grad           FP32[n] device, read (the reduced gradient shard).
 *   grad_scale     NULL, or a device float (4-byte aligned, outside the written
 *                  buffers): g is first multiplied by it, as in
 *                  zero_adam_shard_step_scaled.
 * Per element, with b = hp->momentum and 1-b a binary32 subtraction:
 *   m' = b*m + (1-b)*g;  u = nesterov ? (1-b)*g + b*m' : m';
 *   direction_out = round_to_nearest_even_bf16(u).
 * The averaged form; a form that sums (m' = b*m + g) differs by the factor 1-b
 * in all of m and u, which the orthogonalisation removes.
 * Errors: ZERO_ERR_ARG (NULL, n < 0, overlap, momentum outside [0, 1),
 * nesterov not 0 or 1), ZERO_ERR_ALIGN, ZERO_ERR_SIZE, ZERO_ERR_HIP. */
int zero_muon_momentum(float* momentum, uint16_t* direction_out, const float* grad,
                       const float* grad_scale, int64_t n, const zero_muon_hparams* hp, void* stream);

/* Reduce-scatter and momentum step in one pass: for every owner k exactly
 * zero_reduce_scatter's shard k (grad_acc[k] + red when grad_acc is given),
 * not stored, and zero_muon_momentum's step with it: bit-identical to the two
 * calls, with 8 fewer bytes of HBM traffic per parameter.
 *   rank_grads, rank_weights, n_ranks, numel, n_shards: as zero_reduce_scatter.
 *   momentum       host array of n_shards device pointers, FP32, numel/n_shards each.
 *   direction_out  host array of n_shards device pointers, BF16.
 *   grad_acc       NULL, or a host array of n_shards device pointers, FP32, read.
 * Errors: as zero_reduce_scatter and zero_muon_momentum; outputs must be
 * disjoint from every other buffer. */
int zero_reduce_scatter_muon(const uint16_t* const* rank_grads, const float* rank_weights, int n_ranks,
                             int64_t numel, int n_shards, float* const* momentum,
                             uint16_t* const* direction_out, const float* const* grad_acc,
                             const zero_muon_hparams* hp, void* stream);

/* Bytes of device workspace zero_newton_schulz needs for n_mats matrices of
 * rows x cols.  Errors: ZERO_ERR_ARG (NULL, a negative size), ZERO_ERR_SIZE. */
int zero_newton_schulz_workspace(int64_t n_mats, int64_t rows, int64_t cols, int64_t* bytes_out);

/* Orthogonalise a stack of matrices by Newton-Schulz products.  For each
 * matrix G (rows x cols):
 *   X = G / ||G||_F  (Frobenius norm; a zero matrix stays zero)
 *   for each step's (a, b, c):  A = X X^T;  X = a X + (b A + c A A) X
 *   out = round_to_nearest_even_bf16(scale * X)
 * that is, every singular value s of X becomes a s + b s^3 + c s^5 per step
 * and the singular vectors stay.  The result does not depend on the input's
 * scale.  A matrix holding a NaN or an infinity gives NaN throughout.
 *   in            device, BF16 or FP32 (in_dtype), element (i, j) of matrix q
 *                 at in[q*in_mat_stride + i*in_row_stride + j].  No two
 *                 elements may share a place; matrices may be column ranges
 *                 of one wider buffer.
 *   out           device, BF16, laid out likewise with its own strides.
 *   coefs         host array of 3*steps floats, steps in [1, 16].  They must
 *                 keep the singular values (from [0, 1] on) within
 *                 ZERO_NS_MAX_SIGMA and a step's gain |p(s)/s| within
 *                 ZERO_NS_MAX_GAIN, with room for roundings: a set whose results
 *                 reach values from which the next steps raise them further is
 *                 refused (see below).
 *   scale         finite factor of the result.
 *   workspace     device, 256-byte aligned, workspace_bytes >=
 *                 zero_newton_schulz_workspace's answer; nothing in it carries
 *                 over between calls.
 * Arithmetic: the norm in FP64 (fixed order); the products on the matrix
 * cores with FP16 operands scaled by powers of two and FP32 accumulation, an FP32
 * input as pairs of FP16 values (22 bits).  With the five steps (3.4445, -4.7750,
 * 2.0315) the result, for either input type, is 1.7e-3 to 2.1e-3 of its norm away
 * from the exact one on Gaussian matrices (rounding it to BF16 is 1.66e-3 of that),
 * up to 4e-3 on spectra that fall over three decades, up to 8e-3 on matrices of
 * rank one or with half of the singular values next to nothing, and up to 2e-2 on
 * matrices of a few distinct values, whose roundings agree and add up.  Small
 * matrices, which one compute unit holds, are kept as pairs throughout: there the
 * rounding to BF16 is all of it.
 * Other coefficients raise roundings more or less.  From them alone the library
 * estimates by how much: over singular values from 2^-10 to 1, of the result's
 * singular values, of its singular vectors, and in the directions of singular values
 * next to nothing.  Where the estimate is not far above the five steps' (six of
 * them, cubic steps up to ten, quintics that start near 4 s), errors stay below 2.5e-2.
 * Where it is, every matrix is kept as pairs, for about three times the time: errors
 * are the result's own rounding to BF16, at most 2^-8, and 2^-22 times the estimate.
 * For singular values that is at most 2^-6, or the set is refused with ZERO_ERR_ARG.
 * In the directions of singular values next to nothing it is the sum over the steps t
 * of the products |a_t ... a_last|, whatever that is: many steps that each raise the
 * smallest singular values raise the last bits of X as well.
 * Results are the same bits on every call with the same inputs.
 * Errors: ZERO_ERR_ARG (NULL, negative sizes, in_dtype, steps, coefficients
 * that are not finite, break the bounds or leave no room for roundings, a scale that is not finite,
 * overlapping buffers), ZERO_ERR_ALIGN, ZERO_ERR_SIZE (strides with which
 * elements share a place, sides above ZERO_NS_MAX_SIDE, more than ZERO_NS_MAX_MATS
 * matrices, a small workspace), ZERO_ERR_HIP. */
int zero_newton_schulz(const void* in, int in_dtype, int64_t in_row_stride, int64_t in_mat_stride,
                       uint16_t* out, int64_t out_row_stride, int64_t out_mat_stride, int64_t n_mats,
                       int64_t rows, int64_t cols, const float* coefs, int steps, float scale,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Owner update with the orthogonalised directions, n elements of its shard:
 *   u = o;  if wd != 0: u = o + wd*p;  p' = p - lr*u;
 *   bf16_out = round_to_nearest_even_bf16(p').
 *   master     FP32[n] device, updated in place.
 *   bf16_out   BF16[n] device, written: the new working weights.
 *   update     BF16[n] device, read: the owner's slice of zero_newton_schulz's results.
 *   lr_dev     NULL, or a device float (4-byte aligned, outside the written
 *              buffers) read when the kernel runs, in place of hp->lr: a
 *              captured graph then replays with each step's learning rate.
 * Errors: as zero_muon_momentum. */
int zero_muon_shard_step(float* master, uint16_t* bf16_out, const uint16_t* update, int64_t n,
                         const zero_muon_hparams* hp, const float* lr_dev, void* stream);

/* ---------------------------------------------------------------- a layer's own work
 * Between the gather of a layer's weights and the reduction of its gradients lies
 * the layer's work ([essay] ZeRO-3 的一次完整计算: gather -> forward -> release;
 * gather -> backward -> reduce-scatter -> owner update).  These calls are that of the
 * gated feed-forward block, which holds most of a layer's parameters: it reads the
 * gathered BF16 view and writes the BF16 contributions that zero_reduce_scatter
 * takes.  What the backward pass needs of the forward is kept in 8 bits. */

/* Formats of an 8-bit checkpoint: two's complement whole numbers in [-127, 127], or
 * e4m3 (sign, 4 exponent bits with bias 7, 3 fraction bits; largest value 448). */
enum { ZERO_ACT8_INT8 = 0, ZERO_ACT8_E4M3 = 1 };

/* Activations into 8 bits.  The columns of a row are taken in blocks of
 * ZERO_ACT8_BLOCK (the last one of a row may be shorter).  With a the block's largest magnitude and
 * M = 127 or 448,
 *   e = the least whole number >= -126 with a <= M * 2^e,
 *   code = round_to_nearest_even(x * 2^-e) in the format,  scale = e + 127.
 * The scaling is exact and no value saturates.  A whole number is off by at most
 * 2^-1 * 2^e (a / 127 at most, but for blocks at the least e, which may lose all of
 * a), an e4m3 value by at most 2^-4 of itself (or 2^-10 * 2^e).
 * A block that holds a NaN, an infinity or a magnitude above 127 * 2^121 (e4m3: 448 *
 * 2^119), next to which a code could stand for 2^128, has scale 255 and codes 0.
 *   x             device, BF16 or FP32 (x_dtype), element (i, j) at
 *                 x[i*x_row_stride + j]; aligned to its element.
 *   codes         device, written: rows * cols bytes, row by row, any alignment.
 *   scales        device, written: rows * ceil(cols / ZERO_ACT8_BLOCK) bytes.
 * Errors: ZERO_ERR_ARG (NULL, negative sizes, x_dtype, format, overlapping buffers),
 * ZERO_ERR_ALIGN, ZERO_ERR_SIZE (a row stride below cols or above ZERO_ACT8_MAX_COLS, more than
 * ZERO_ACT8_MAX_COLS columns, or than ZERO_ACT8_MAX_VALUES values with every row's last
 * block filled up), ZERO_ERR_HIP. */
int zero_act8_save(const void* x, int x_dtype, int64_t x_row_stride, int64_t rows, int64_t cols, int format,
                   uint8_t* codes, uint8_t* scales, void* stream);

/* The values of a checkpoint: code * 2^(scale - 127), exact in FP32 and, from 2^-126 on,
 * in BF16 (below, rounded to nearest even); a block with scale 255 reads as NaN.
 *   out           device, written, BF16 or FP32 (out_dtype), laid out as
 *                 zero_act8_save's x.
 * Errors: as zero_act8_save. */
int zero_act8_load(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int format, void* out,
                   int out_dtype, int64_t out_row_stride, void* stream);

/* Activations of the feed-forward block: x sigma(x); x sigma(2 sqrt(2/pi) (x + 0.044715 x^3)),
 * which is GELU with tanh; max(x, 0), whose derivative at 0 is taken as 0. */
enum { ZERO_FFN_SILU = 0, ZERO_FFN_GELU = 1, ZERO_FFN_RELU = 2 };

/* What a forward pass keeps for the backward pass: the block's input x
 * [tokens, model], and g = x Wg^T and u = x Wu^T [tokens, hidden], each as
 * zero_act8_save lays it out.  model + 2 hidden bytes per token and 1/32 more, where
 * BF16 values of x, g, u and h would be 2 model + 6 hidden. */
typedef struct zero_ffn_checkpoint {
  uint8_t *x_codes, *x_scales, *gate_codes, *gate_scales, *up_codes, *up_scales;
  int32_t format;
} zero_ffn_checkpoint;

/* Bytes of workspace with which zero_ffn_forward, or with ZERO_FFN_BACKWARD
 * zero_ffn_backward, takes any count of tokens up to `tokens`.  (A call may need more
 * than one of more tokens: sums of few rows are shared out, with room for the parts.)
 * Weights that are not 16-byte aligned need ZERO_FFN_UNALIGNED (room for aligned
 * copies; sizes that are no multiples of 64 have that room anyway).
 * Errors: ZERO_ERR_ARG (NULL, unknown flags, tokens < 0, a side < 1), ZERO_ERR_SIZE
 * (sizes above ZERO_FFN_MAX_TOKENS, ZERO_FFN_MAX_SIDE, or activations that
 * zero_act8_save would refuse). */
int zero_ffn_workspace(int64_t tokens, int64_t model, int64_t hidden, int flags, int64_t* bytes_out);

/* Gated feed-forward block, forward:
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) * u,  y = h Wd^T.
 *   x, y          device BF16, element (t, j) at x[t*x_row_stride + j], 2-byte aligned.
 *                 With one row stride they may be columns of one buffer, side by side.
 *   w_gate, w_up  device BF16 [hidden, model], w_down [model, hidden], contiguous:
 *                 slices of the gathered view of a layer.
 *   save          host, or NULL: the checkpoint's buffers, written.
 *   workspace     device, 256-byte aligned, workspace_bytes >= zero_ffn_workspace's
 *                 answer for as many tokens or more; nothing in it carries over
 *                 between calls.  Calls that may run at the same time (streams,
 *                 captured graphs) need one each.
 * Arithmetic: products of BF16 values summed in FP32 on the matrix cores; act in
 * FP32; g and u go into the checkpoint as summed, h is rounded to BF16 (the type the
 * second product takes), y is rounded to BF16.  Results are the same bits on every
 * call with the same inputs, y whether a checkpoint is written or not.
 * tokens = 0 launches nothing.
 * Errors: ZERO_ERR_ARG (NULL, negative sizes, activation, format, overlapping
 * buffers: nothing written may overlap anything else), ZERO_ERR_ALIGN, ZERO_ERR_SIZE
 * (limits, a row stride below model or above ZERO_FFN_MAX_STRIDE, a small
 * workspace), ZERO_ERR_HIP. */
int zero_ffn_forward(const uint16_t* x, int64_t x_row_stride, int64_t tokens, int64_t model, int64_t hidden,
                     const uint16_t* w_gate, const uint16_t* w_up, const uint16_t* w_down, int activation,
                     uint16_t* y, int64_t y_row_stride, const zero_ffn_checkpoint* save, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* Backward, from a checkpoint's values of x, g and u:
 *   dh = dy Wd,  dg = dh * u * act'(g),  du = dh * act(g),  h = act(g) * u,
 *   dx = dg Wg + du Wu,  d_gate = dg^T x,  d_up = du^T x,  d_down = dy^T h.
 *   dy, dx        device BF16 with row strides, as x and y; dx may be NULL (not wanted).
 *   saved         host: the checkpoint's buffers, read.
 *   d_gate, d_up  device BF16 [hidden, model], d_down [model, hidden], contiguous,
 *                 written: slices of a rank's gradient contribution.
 * Arithmetic as in the forward pass; dg, du and h are rounded to BF16 between the
 * products.  tokens = 0: the gradients are zeros (a rank without tokens contributes
 * nothing), and only they are touched.
 * Errors: as zero_ffn_forward, and ZERO_ERR_ARG for a NULL checkpoint. */
int zero_ffn_backward(const uint16_t* dy, int64_t dy_row_stride, int64_t tokens, int64_t model, int64_t hidden,
                      const zero_ffn_checkpoint* saved, const uint16_t* w_gate, const uint16_t* w_up,
                      const uint16_t* w_down, int activation, uint16_t* dx, int64_t dx_row_stride, uint16_t* d_gate,
                      uint16_t* d_up, uint16_t* d_down, void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- host-offloaded gradient shard */

/* Two device slots stream a gradient shard that lives in pinned host memory
 * ([blog] 分片放到 CPU：两个缓冲就够): chunk c of the shard uses slot c % 2.
 *
 * Caller-owned buffers, all given at creation:
 *   host_shard_pinned  FP32[shard_numel] pinned host memory (hipHostMalloc,
 *                      or a pinned torch tensor): the accumulator.
 *   slot_contrib[s]    device BF16 buffer of n_ranks*chunk_numel values: rank
 *                      r's contribution to the chunk in slot s starts at
 *                      slot_contrib[s] + r*chunk_numel (a partial last chunk
 *                      uses the first elements of each rank's range).
 *   slot_f32[s]        device FP32 buffer of chunk_numel values (staging).
 * The handle owns two side streams (host-to-device, device-to-host) and
 * events only.
 *
 * zero_offload_stream(op = ZERO_OFFLOAD_REDUCE, chunk c, micro_batch mb):
 *   the caller has written chunk c's contributions into slot_contrib[c % 2] on
 *   compute_stream.  mb == 0: staging = red(c).  mb > 0: the host chunk is
 *   copied in, staging = staging + red(c).  Then staging is copied to the
 *   host chunk asynchronously.  red is zero_reduce_scatter's reduction with
 *   rank_weights.  When the call returns the caller may write the next
 *   contributions for slot c % 2 on compute_stream.
 * zero_offload_stream(op = ZERO_OFFLOAD_ADAM, chunk c):
 *   the host chunk is copied into slot_f32[c % 2] and zero_adam_shard_step runs
 *   on it with the chunk's elements of master/exp_avg/exp_avg_sq/bf16_out
 *   (device pointers to the whole shard).
 * zero_offload_stream(op = ZERO_OFFLOAD_REDUCE_ADAM, chunk c, micro_batch mb):
 *   the last micro-batch of chunk c fused with its update: the host chunk
 *   (micro-batches 0..mb-1) is copied in when mb > 0, and the reduction of the
 *   slot is added to it and applied by zero_reduce_scatter_adam's update
 *   without a copy back: the final accumulated gradient never crosses the
 *   link (16 fewer link bytes per parameter and step).  Results are
 *   bit-identical to REDUCE for mb followed by ADAM; the host chunk then holds
 *   micro-batches 0..mb-1 only.
 * zero_offload_sync: waits for every queued copy and kernel of the handle; the
 *   host shard may be read after it returns.
 * zero_offload_destroy: waits for the handle's copies and kernels, then frees
 *   its streams, events and the handle itself (never the caller's buffers);
 *   NULL is a no-op.  Returns ZERO_ERR_HIP if a wait failed (the handle is
 *   freed all the same).
 * compute_stream may change from one call to the next: the handle orders its
 * own copies and kernels on each slot by events.  Ordering the writes into
 * slot_contrib after the kernel that last read that slot stays the caller's
 * (automatic when both run on one stream).
 * Errors: ZERO_ERR_ARG / ZERO_ERR_ALIGN / ZERO_ERR_SIZE for bad arguments
 * (ZERO_ERR_ARG also for a host shard that is not pinned host memory)
 * (ZERO_ERR_SIZE also for more than ZERO_OFFLOAD_MAX_CHUNKS chunks: the handle
 * keeps two events per chunk, or when the handle's host memory cannot be
 * allocated), ZERO_ERR_STATE for a chunk out of range, a REDUCE or REDUCE_ADAM
 * with mb > 0 whose micro-batch mb - 1 is not the chunk's last one, or an ADAM
 * for a chunk with no accumulation: never reduced, or already consumed by an
 * ADAM or REDUCE_ADAM (after which the chunk starts again at mb 0);
 * ZERO_ERR_HIP on runtime failures. */
typedef struct zero_offload zero_offload;
enum { ZERO_OFFLOAD_REDUCE = 0, ZERO_OFFLOAD_ADAM = 1, ZERO_OFFLOAD_REDUCE_ADAM = 2 };

int zero_offload_create(int n_ranks, int64_t shard_numel, int64_t chunk_numel,
                        float* host_shard_pinned, uint16_t* const slot_contrib[2],
                        float* const slot_f32[2], zero_offload** out);
int zero_offload_stream(zero_offload* h, int op, int64_t chunk, int micro_batch,
                        const float* rank_weights, float* master, float* exp_avg,
                        float* exp_avg_sq, uint16_t* bf16_out, const zero_adam_hparams* hp,
                        void* compute_stream);
int zero_offload_sync(zero_offload* h);
int zero_offload_destroy(zero_offload* h);

/* ---------------------------------------------------------------- diagnostics */
const char* zero_status_string(int status);
const char* zero_last_error(void);
/* 1 if the last device call took the 16-byte vector path, 0 for the scalar
 * path (used by tests to cover both paths). */
int zero_last_path_vectorized(void);

/* 1 when the device entry points emit ROCTX ranges (one per call, named after
 * the call): set ZERO_ROCTX=1 in the environment before the library's first
 * call; ROCm's roctx library is then loaded at run time, and rocprofv3
 * --marker-trace records the ranges.  0 otherwise (no cost). */
int zero_tracing_enabled(void);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_H */
