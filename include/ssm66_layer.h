/*
 * ssm66_layer.h -- C ABI of a gated linear recurrence and of what stands around
 * a mixer in a layer, in the same library as ssm66.h and with its conventions:
 * caller-owned device pointers, dense row-major tensors, no allocation, every
 * call asynchronous on the caller's stream (of the current device), arguments
 * checked before any HIP call, the status codes and io dtypes of ssm66.h,
 * float32 states and parameters in every mode.
 *
 *   ssm_gated_scan_fwd, ssm_gated_scan_bwd, ssm_gated_scan_step
 *       a recurrence of one state per channel whose decay and input are gated
 *       by the data: sequences, gradients, one token.
 */
#ifndef SSM66_LAYER_H
#define SSM66_LAYER_H

#include "ssm66.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The gated linear recurrence.  For each entry and channel,
 *   v_t = decay[c] sigmoid(r_t),   a_t = exp(-v_t),
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t.
 *   x, r, i, y : (batch, seqlen, dim), io dtype; r and i are the gates before
 *                their sigmoid
 *   decay      : (dim) float32, finite, not negative; 0 keeps the state
 *   h0         : (batch, dim) float32, the state before token 0, or NULL (zero)
 *   seq_lens   : (batch) int32 or NULL: as for ssm_scan_fwd_ex -- tokens at or
 *                past a length are padding, whatever they hold: y = 0 there and
 *                the state is the one after the last real token
 *   reset      : (batch, seqlen) uint8 or NULL: the state is zeroed before a
 *                flagged token (a document starts there)
 *   last_state : (batch, dim) float32, or NULL; must not overlap h0
 *   states     : (batch, ceil(seqlen / 128), dim) float32, or NULL: the state
 *                before every 128th token, which ssm_gated_scan_bwd takes
 * Tensors are aligned to their element size (bf16 to 4 bytes, with dim even, is
 * fastest); outputs and workspace overlap no input.  dim at most 2^24, batch *
 * ceil(dim / 64) * ceil(seqlen / 128) below 2^31 and seqlen below 2^31 - 128
 * (else SSM_ERR_UNSUPPORTED).  Zero batch or dim is a no-op; seqlen == 0 copies
 * h0 (or zero) to last_state.
 * workspace: ssm_gated_scan_workspace_size(..., 0, 0) bytes, 256-byte aligned,
 * contents not needed before or after (NULL where the size is 0).
 * Values are not checked: a NaN or infinity in a real token reaches the later
 * tokens of its document, no other document and no other channel.  Repeated
 * calls give identical bits.
 */
size_t ssm_gated_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int backward,
                                     int need_ddecay);
int ssm_gated_scan_fwd(const void* x, const void* r, const void* i, const float* decay,
                       const float* h0, const int32_t* seq_lens, const uint8_t* reset, void* y,
                       float* last_state, float* states, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, void* stream);

/*
 * Gradients of ssm_gated_scan_fwd, from its inputs and the states it kept (h0 is
 * the first of them).
 *   dy         : (batch, seqlen, dim), io dtype
 *   dlast      : (batch, dim) float32, the gradient of last_state, or NULL (zero)
 *   dx, dr, di : like x; zero at padding
 *   ddecay     : (dim) float32, or NULL (not a number where decay is 0: the root
 *                has no derivative there)
 *   dh0        : (batch, dim) float32, or NULL; must not overlap dlast
 * Outputs are overwritten.  workspace: ssm_gated_scan_workspace_size(..., 1,
 * ddecay != NULL) bytes.  Alignment and limits as for ssm_gated_scan_fwd; zero
 * batch writes zeros to ddecay.  All sums are taken in a fixed order: repeated
 * calls give identical bits.
 */
int ssm_gated_scan_bwd(const void* x, const void* r, const void* i, const float* decay,
                       const float* states, const int32_t* seq_lens, const uint8_t* reset,
                       const void* dy, const float* dlast, void* dx, void* dr, void* di,
                       float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, void* stream);

/*
 * One token against a state cache (batch, dim) float32, updated in place; x, r,
 * i, y: (batch, dim), io dtype; y may be any of them.  dim at most 2^24.
 */
int ssm_gated_scan_step(float* state, const void* x, const void* r, const void* i,
                        const float* decay, void* y, int64_t batch, int64_t dim, int io_dtype,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM66_LAYER_H */
