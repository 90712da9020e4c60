/*
 * ssm66_layer.h -- C ABI of a gated linear recurrence and of what stands around
 * a mixer in a layer, in the same library as ssm66.h and with its conventions:
 * caller-owned device pointers, dense row-major tensors, no allocation, every
 * call asynchronous on the caller's stream (of the current device), arguments
 * checked before any HIP call, the status codes and io dtypes of ssm66.h,
 * float32 states and parameters in every mode.  An output shares memory with an
 * input only where that is said ("may be"), from the first byte to the last, and
 * with no other output and no workspace: else SSM_ERR_FLAG.
 *
 *   ssm_gated_scan_fwd, ssm_gated_scan_bwd, ssm_gated_scan_step
 *       a recurrence of one state per channel whose decay and input are gated
 *       by the data: sequences, gradients, one token.
 *   ssm_add_norm_fwd, ssm_add_norm_bwd
 *       a residual, a dropped-out branch and the layer or RMS norm of their sum.
 *   ssm_dropout
 *       dropout from a counter-based generator, the mask never stored.
 *   ssm_rotary
 *       rotary positions of queries and keys, and their gradients.
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
 *   decay      : (dim) float32, 0 to 1e30 (v of 1e38 overflows in its products);
 *                0 keeps the state
 *   h0         : (batch, dim) float32, the state before token 0, or NULL (zero)
 *   seq_lens   : (batch) int32 or NULL: as for ssm_scan_fwd_ex -- tokens at or
 *                past a length are padding, whatever they hold: y = 0 there and
 *                the state is the one after the last real token
 *   reset      : (batch, seqlen) uint8 or NULL: the state is zeroed before a
 *                flagged token (a document starts there)
 *   last_state : (batch, dim) float32, or NULL; must not overlap h0
 *   states     : (batch, ceil(seqlen / 64), dim) float32, or NULL: the state
 *                before every 64th token, which ssm_gated_scan_bwd takes
 * Tensors are aligned to their element size (to 128 bytes, and rows of as many or
 * a multiple, is fastest).  No output may be an input (two blocks may read one
 * channel, and all blocks of a row read h0).  dim at most 2^24, batch * ceil(dim /
 * 64) * ceil(seqlen / 64) below 2^31 and seqlen at most 2^31 - 256 (else
 * SSM_ERR_UNSUPPORTED).  Zero batch or dim is a no-op; seqlen == 0 copies h0 (or
 * zero) to last_state.
 * workspace: ssm_gated_scan_workspace_size(..., 0, 0) bytes, 256-byte aligned,
 * contents not needed before or after (NULL where the size is 0).  It serves one
 * call at a time: its blocks wait for one another through it, and two calls that
 * run at once on one workspace could wait for ever.
 * Values are not checked: a NaN or infinity in a real token reaches the later
 * tokens of its document (an infinite state stays infinite; a bfloat16 call makes
 * it a NaN at a token whose v is over 87, where a is 0 in float32), no other
 * document and no other channel.  Repeated calls give identical bits.
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
 * Outputs are overwritten; none may be an input.  workspace:
 * ssm_gated_scan_workspace_size(..., 1, ddecay != NULL) bytes.  Alignment and
 * limits as for ssm_gated_scan_fwd; zero batch or seqlen writes zeros to ddecay.
 * All sums are taken in a fixed order: repeated calls give identical bits.
 */
int ssm_gated_scan_bwd(const void* x, const void* r, const void* i, const float* decay,
                       const float* states, const int32_t* seq_lens, const uint8_t* reset,
                       const void* dy, const float* dlast, void* dx, void* dr, void* di,
                       float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, void* stream);

/*
 * One token against a state cache (batch, dim) float32, updated in place; x, r,
 * i, y: (batch, dim), io dtype; y may be any of x, r and i.  dim at most 2^24.
 */
int ssm_gated_scan_step(float* state, const void* x, const void* r, const void* i,
                        const float* decay, void* y, int64_t batch, int64_t dim, int io_dtype,
                        void* stream);

/*
 * Random numbers of ssm_dropout and the add_norm calls: Philox4x32 with ten
 * rounds under the key rng[0] (low word first).  Value e of a tensor (its place
 * in row-major order) takes word e % 4 of the block with the 128-bit counter
 * (e / 4, rng[1] + site), low words first; it is dropped where word < p 2^32
 * (rounded down), else multiplied with 1 / (1 - p).  rng lies in device memory,
 * so that a captured graph draws anew when the program moves rng[1] on; a
 * backward call takes the rng and site of its forward.
 *   rng  : (2) int64, device: seed and offset; may be NULL where p is 0
 *   site : added to the offset: one number for each place that drops
 *   p    : 0 <= p < 1
 *
 * Dropout: y = dropout(x) + residual (NULL: none).
 *   x           : (n) io_dtype
 *   residual, y : (n) out_dtype; y may be x (of one type) or residual, or both
 * The gradient of x is ssm_dropout of dy, without a residual, from out_dtype to
 * io_dtype.  Tensors are aligned to their element size (16 bytes is fastest);
 * zero n is a no-op.  A dropped value counts as 0 whatever it is.
 */
int ssm_dropout(const void* x, const void* residual, const int64_t* rng, int64_t site, float p,
                void* y, int64_t n, int io_dtype, int out_dtype, void* stream);

/* norms of ssm_add_norm_fwd */
#define SSM_NORM_LAYER 0
#define SSM_NORM_RMS 1

/*
 * A residual stream, a branch that joins it, and the norm of their sum:
 *   h = residual + dropout(x)   (rounded to h's type; the norm is of that),
 *   y = (h - mean) / sqrt(var + eps) weight + bias       (SSM_NORM_LAYER),
 *   y = h / sqrt(mean of squares + eps) weight + bias    (SSM_NORM_RMS)
 * over each row, the variance over the same values (not one less).
 *   x, y         : (rows, dim), io_dtype
 *   residual, h  : (rows, dim), h_dtype, which is io_dtype or SSM_F32; either
 *                  may be NULL (no residual; h not kept).  h may be residual,
 *                  or x where they are of one type
 *   weight, bias : (dim) float32, or NULL (one, zero)
 *   mean, rstd   : (rows) float32, or NULL: what ssm_add_norm_bwd takes (mean
 *                  is not written by the RMS norm)
 * y may be x.  dim at most 16384 (else SSM_ERR_UNSUPPORTED).  Squares are summed
 * in float32: values stay below 1e17 (a sum past 3e38 makes rstd 0).  Tensors are
 * aligned to their element size (to 16 bytes, and with dim a multiple of 8, is
 * fastest).  Zero rows is a no-op.
 */
int ssm_add_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                     int norm, float eps, float p, const int64_t* rng, int64_t site, void* y,
                     void* h, float* mean, float* rstd, int64_t rows, int64_t dim, int io_dtype,
                     int h_dtype, void* stream);

/*
 * Gradients of ssm_add_norm_fwd, from the h, mean and rstd it wrote (without a
 * residual and with p = 0, h is x).
 *   dy             : (rows, dim), io_dtype
 *   dh             : (rows, dim), h_dtype, the gradient of h from elsewhere, or
 *                    NULL (zero)
 *   dx             : (rows, dim), io_dtype
 *   dresidual      : (rows, dim), h_dtype, or NULL
 *   dweight, dbias : (dim) float32, or NULL
 * Outputs are overwritten; dx and dresidual may each be dy or dh, of their type.
 * workspace: ssm_add_norm_workspace_size(...) bytes, 256-byte aligned (NULL and 0
 * where neither dweight nor dbias is asked for).  Zero rows writes zeros to
 * dweight and dbias.  All sums are taken in a fixed order: repeated calls give
 * identical bits.
 */
size_t ssm_add_norm_workspace_size(int64_t rows, int64_t dim);
int ssm_add_norm_bwd(const void* h, const void* dy, const void* dh, const float* weight, int norm,
                     const float* mean, const float* rstd, float p, const int64_t* rng,
                     int64_t site, void* dx, void* dresidual, float* dweight, float* dbias,
                     void* workspace, size_t workspace_bytes, int64_t rows, int64_t dim,
                     int io_dtype, int h_dtype, void* stream);

/*
 * Rotary positions.  Pair j of each head is turned by the angle t = position
 * freqs[j] and scaled:
 *   (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t),
 * a and b the elements 2j and 2j + 1 of the head (interleaved != 0) or j and
 * j + rot / 2.  The elements from rot on are copied.
 *   q, q_out  : (batch, seqlen, heads, dim), io dtype
 *   k, k_out  : (batch, seqlen, kheads, dim), or NULL with kheads = 0
 *   freqs     : (rot / 2) float32, taken as exact (the angle is formed in 64 bits)
 *   positions : (batch, seqlen) int32, or NULL: 0 .. seqlen - 1 in each entry
 *   inverse   : nonzero turns by -t, which is the gradient of the call without
 * q_out may be q and k_out may be k.  rot is even, 2 <= rot <= dim.  Tensors are
 * aligned to their element size (16 bytes, with dim and rot -- halves: rot / 2 --
 * multiples of 16 bytes, is fastest).  heads, kheads and dim at most 2^20, batch
 * * seqlen * (heads + kheads) * dim below 2^38, seqlen below 2^31 (else
 * SSM_ERR_UNSUPPORTED).  Zero batch or seqlen is a no-op.
 */
int ssm_rotary(const void* q, const void* k, const float* freqs, const int32_t* positions,
               float mscale, int interleaved, int inverse, void* q_out, void* k_out, int64_t batch,
               int64_t seqlen, int64_t heads, int64_t kheads, int64_t dim, int64_t rot,
               int io_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM66_LAYER_H */
