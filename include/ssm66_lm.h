/*
 * ssm66_lm.h -- C ABI of the operators around a linear-attention layer, in the
 * same library as ssm66.h and with its conventions: caller-owned device
 * pointers, dense row-major tensors, no allocation, every call asynchronous on
 * the caller's stream, arguments checked before any HIP call, the status codes
 * and io dtypes of ssm66.h, float32 states and parameters in every mode.
 *
 *   ssm_linattn_fwd, ssm_linattn_bwd, ssm_linattn_step
 *       linear attention with a decay for each head: prompts, gradients, one
 *       token.
 *   ssm_group_norm_fwd, ssm_group_norm_bwd
 *       group norm, channels last, with an activation and a gate.
 *   ssm_clip_grad_norm
 *       the global norm of many gradients, and the gradients clipped to it.
 */
#ifndef SSM66_LM_H
#define SSM66_LM_H

#include "ssm66.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay for each head.  Head h of `nheads` reads the
 * keys of key head h / (nheads / kheads), and with lam = exp(log_decay[h])
 *   S_t = lam S_{t-1} + v_t k_t^T        (S: dv x dk),
 *   o_t = scale S_t q_t.
 *   q, k       : (batch, seqlen, kheads, dk), io dtype
 *   v, o       : (batch, seqlen, nheads, dv), io dtype
 *   log_decay  : (nheads) float32; the log of the factor per token, 0 = keep
 *                everything, -inf = keep nothing
 *   h0         : (batch, nheads, dv, dk) float32, the state before token 0, or
 *                NULL (zero)
 *   seq_lens   : (batch) int32 or NULL: as for ssm_scan_fwd_ex -- tokens at or
 *                past a length are padding, whatever they hold: o = 0 there and
 *                the state is the one after the last real token
 *   reset      : (batch, seqlen) uint8 or NULL: the state is zeroed before a
 *                flagged token (a document starts there)
 *   last_state : (batch, nheads, dv, dk) float32, or NULL; must not overlap h0
 * kheads divides nheads; dk and dv are multiples of 8, at most 256; q, k, v
 * and o are 16-byte aligned, and so are h0 and last_state; nheads * dv and
 * kheads * dk at most 2^22, batch * nheads below 2^21, seqlen at most 2^29 - 64
 * (else SSM_ERR_UNSUPPORTED).  Zero batch or nheads is a no-op; seqlen == 0
 * copies h0 (or zero) to last_state.
 * workspace: ssm_linattn_fwd_workspace_size(...) bytes, 256-byte aligned,
 * contents not needed before or after (NULL where the size is 0).  Outputs and
 * workspace overlap no input.
 * Values are not checked.  A NaN or infinity in a real token reaches all outputs
 * of its own chunk of 64 tokens (tokens before it and other documents too), the
 * later ones of its document and the state, if the document lasts to its end; no
 * other.  float32 values of a magnitude over 3.396e38 (half a unit past bf16's
 * largest) count as infinities.  Repeated calls give identical bits.
 */
size_t ssm_linattn_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads,
                                      int64_t kheads, int64_t dk, int64_t dv, int io_dtype);
int ssm_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const float* h0, const int32_t* seq_lens, const uint8_t* reset,
                    void* o, float* last_state, void* workspace, size_t workspace_bytes,
                    int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                    int64_t dv, int io_dtype, void* stream);

/*
 * Gradients of ssm_linattn_fwd, from its inputs (the states are recomputed).
 *   do_        : (batch, seqlen, nheads, dv), io dtype
 *   dlast      : (batch, nheads, dv, dk) float32, the gradient of last_state,
 *                or NULL (zero)
 *   dq, dk_, dv_ : like q, k, v (dq and dk_ summed in float32 over the heads
 *                that share a key head, rounded once); zero at padding
 *   dlog_decay : (nheads) float32, or NULL
 *   dh0        : (batch, nheads, dv, dk) float32, or NULL
 * Outputs are overwritten.  A token sees no gradient from after the next
 * document start.  workspace: ssm_linattn_bwd_workspace_size(...) bytes,
 * 256-byte aligned (need_dlog_decay says whether dlog_decay is asked for).
 * Alignment and limits as for ssm_linattn_fwd, and nheads * dk at most 2^22.
 * All sums are taken in a fixed order: repeated calls give identical bits.
 */
size_t ssm_linattn_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads,
                                      int64_t kheads, int64_t dk, int64_t dv,
                                      int need_dlog_decay, int io_dtype);
int ssm_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const float* h0, const int32_t* seq_lens, const uint8_t* reset,
                    const void* do_, const float* dlast, void* dq, void* dk_, void* dv_,
                    float* dlog_decay, float* dh0, void* workspace, size_t workspace_bytes,
                    int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                    int64_t dv, int io_dtype, void* stream);

/*
 * One token against a state cache (batch, nheads, dv, dk) float32, updated in
 * place: S = lam S + v k^T, o = scale S q.  q, k: (batch, kheads, dk);
 * v, o: (batch, nheads, dv), io dtype.  dk is a multiple of 8, at most 256; dv
 * any positive size up to 2^30, batch * nheads * ceil(dv / 4) below 2^31 (else
 * SSM_ERR_UNSUPPORTED); state, q and k are 16-byte aligned, v and o to their
 * element size.
 */
int ssm_linattn_step(float* state, const void* q, const void* k, const void* v,
                     const float* log_decay, float scale, void* o, int64_t batch,
                     int64_t nheads, int64_t kheads, int64_t dk, int64_t dv, int io_dtype,
                     void* stream);

/* activations of ssm_group_norm_fwd */
#define SSM_ACT_NONE 0
#define SSM_ACT_SILU 1

/*
 * Group norm over channels-last tensors.  Entry n and group g normalise over
 * the rows and the channels / groups channels of the group together:
 *   xh = (x - mean) / sqrt(var + eps),  u = xh weight[c] + bias[c],
 *   y = act(u) silu(z)
 * with the variance over the same values (not one less).  rows == 1 is the
 * norm of each token's heads: the batch holds the tokens.
 *   x, z, y      : (batch, rows, channels), io dtype; z may be NULL (no gate)
 *   weight, bias : (channels) float32, or NULL (one, zero)
 *   mean, rstd   : (batch, groups) float32, or NULL: what ssm_group_norm_bwd
 *                  takes
 * groups divides channels; channels at most 2^22, batch * groups below 2^31
 * (else SSM_ERR_UNSUPPORTED).  Tensors are aligned to their element size (to 16
 * bytes, and with channels / groups a multiple of 16 bytes, is fastest).  y may
 * be x or z.  Zero batch or rows is a no-op.
 * workspace: ssm_group_norm_workspace_size(..., 0, ...) bytes, 256-byte
 * aligned.  Repeated calls give identical bits.
 */
size_t ssm_group_norm_workspace_size(int64_t batch, int64_t rows, int64_t channels,
                                     int64_t groups, int backward, int io_dtype);
int ssm_group_norm_fwd(const void* x, const float* weight, const float* bias, const void* z,
                       int act, float eps, void* y, float* mean, float* rstd, void* workspace,
                       size_t workspace_bytes, int64_t batch, int64_t rows, int64_t channels,
                       int64_t groups, int io_dtype, void* stream);

/*
 * Gradients of ssm_group_norm_fwd, from its inputs and the mean and rstd it
 * wrote.
 *   dy, dx, dz     : (batch, rows, channels), io dtype; dz is written where z
 *                    is given
 *   dweight, dbias : (channels) float32, or NULL
 * Outputs are overwritten and overlap no input.  workspace:
 * ssm_group_norm_workspace_size(..., 1, ...) bytes, 256-byte aligned.  Zero
 * batch or rows writes zeros to dweight and dbias.
 */
int ssm_group_norm_bwd(const void* x, const float* weight, const float* bias, const void* z,
                       int act, const float* mean, const float* rstd, const void* dy, void* dx,
                       float* dweight, float* dbias, void* dz, void* workspace,
                       size_t workspace_bytes, int64_t batch, int64_t rows, int64_t channels,
                       int64_t groups, int io_dtype, void* stream);

/*
 * The global norm of many gradients, and the gradients clipped to it:
 *   norm = sqrt(sum of the squares of all values of all tensors),
 *   outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)).
 *   grads, outs : HOST arrays of ntensors device pointers; outs[i] may be
 *                 grads[i] (in place), and overlaps no other tensor
 *   counts      : HOST array of element counts (zero is fine)
 *   io_dtypes   : HOST array, SSM_F32 or SSM_BF16 for each tensor
 *   norm        : one float32, device memory
 * The host arrays are read before the call returns.  Squares are added in
 * float64.  A norm that is infinite gives a factor of 0, a NaN spreads to all
 * outputs.  max_norm >= 0.  workspace: ssm_clip_grad_norm_workspace_size(
 * ntensors) bytes, 256-byte aligned.  Repeated calls give identical bits.
 */
size_t ssm_clip_grad_norm_workspace_size(int64_t ntensors);
int ssm_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts,
                       const int32_t* io_dtypes, int64_t ntensors, float max_norm, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM66_LM_H */
