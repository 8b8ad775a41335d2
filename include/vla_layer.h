/*
 * vla_layer.h -- operators of libvla_gb300.so around the recurrence of vla.h:
 * linear attention with a decay per head and the gated delta rule (prompt,
 * gradient, single token), the norm and position rotation of queries and keys and
 * the layer norm of each head's readout with their gradients, and a quantised
 * cache of the heads' states.
 *
 * Conventions as in vla.h: device pointers owned by the caller, `stream` a
 * cudaStream_t as void*, calls asynchronous on it, argument errors returned at
 * once, head dimensions d in {32, 64, 96, 128} (else VLA_ERR_UNSUPPORTED),
 * states in fp32, sums and statistics in fp32. Two things differ. Sequences may
 * have any strides (vla_seq), so that a projection's [B, T, H, d] output is read in
 * place. And results that are sequences (o, y, the gradients) have the inputs'
 * type, rounded at the end; what bf16 calls of vla_decay_*() and vla_delta_*()
 * round before that stands there.
 *
 * An output of a call overlaps neither itself nor an input nor another output
 * (nor the call's scratch), except in place where an entry point says so: blocks
 * of a call read what others write. Rows that lie between those of another array
 * do not overlap it. Checked: VLA_ERR_INVALID_ARG.
 *
 * `status` is the 256-byte status record that the workspace of vla_forward()
 * begins with (zero-filled before the first use, 16-byte aligned); several
 * calls and streams may share it. vla_get_last_device_status(status, ...)
 * reads and clears it. NULL: nothing is recorded.
 */
#ifndef VLA_GB300_LAYER_H
#define VLA_GB300_LAYER_H

#include "vla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [B, H, T, d] sequence: element (b, h, t, i) is data[b * stride_b +
 * h * stride_h + t * stride_t + i], strides in elements. data is 16-byte
 * aligned; the strides of dimensions longer than 1 are positive multiples of
 * 16 bytes (else VLA_ERR_INVALID_ARG). */
typedef struct {
    const void* data;
    long long stride_b, stride_h, stride_t;
} vla_seq;

/* The same for an output. */
typedef struct {
    void* data;
    long long stride_b, stride_h, stride_t;
} vla_seq_out;

/* ---- linear attention with a decay per head --------------------------------
 *
 *   S_t = l S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   l = exp(log_decay[h])
 *
 * S has the layout of vla.h's states ([B, H, d, d], S[i][j] maps key
 * coordinate j to output coordinate i). log_decay: [H] float32; 0 gives
 * the plain cumulative state, -inf forgets everything before the token,
 * positive values are taken as they are: the state grows, and results that
 * overflow are Inf or NaN. (A head that grows by more than a factor of two a
 * token in bf16, or four in fp32, is computed a token at a time.) It is a
 * constant of the layer like lambda0 of vla_forward(): no gradient is formed
 * for it.
 *
 * lengths: NULL, or [B] int32 on the device: sequence b has
 * min(max(lengths[b], 0), T) tokens. Rows of o (or of the gradients) behind
 * them are written as zero, whatever the inputs hold there, and the final
 * state is the one after the sequence's own last token.
 *
 * Rounding. fp32 calls and bf16 calls of up to 8 tokens: fp32 throughout. bf16
 * calls of more tokens: the final states as in fp32; on the way to o, dq, dk and
 * dv the products of pairs of tokens, and the state as the tokens of a chunk of 64
 * find it, are rounded to bf16 (a term meets one of the two, at most 2^-8 of it)
 * and summed in fp32. Errors are then about 2.35e-3 of a row's size, where
 * rounding the exact result to bf16 gives 1.65e-3.
 *
 * A token's NaN or Inf reaches the results that depend on it, as the formulas
 * have it, and no others: no earlier row of o or dq, no later one of dk or dv.
 * One in an output or a final state sets VLA_ERR_NONFINITE in the
 * status record; a bounded in-kernel wait that ran out VLA_ERR_TIMEOUT. */

/* Device scratch a call needs (0 when it needs none, or for sizes the call
 * refuses), for the current device; backward: nonzero for vla_decay_backward().
 * 256-byte aligned, one call's own: calls that may overlap need separate ones. */
size_t vla_decay_scratch_bytes(int B, int H, int T, int d, int backward);

/* The recurrence over T tokens. S0: [B, H, d, d] float32 or NULL for 0;
 * S_out: [B, H, d, d] float32, required, may be S0. T == 0 copies the initial
 * state (q, k, v, o may then be NULL). */
vla_status vla_decay_forward(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H,
                             int T, int d, const float* log_decay, float scale, const int* lengths, const float* S0,
                             const vla_seq_out* o, float* S_out, void* scratch, size_t scratch_bytes, void* status,
                             void* stream);

/* Reverse mode of vla_decay_forward(): from dO = dL/do and dS_T = dL/dS_out
 * (NULL: zero) the gradients dq, dk, dv and, unless NULL, dS0 = dL/dS0:
 *   dq_t = scale S_t^T dO_t,
 *   R_n = dS_T + scale dO_n q_n^T for a sequence's last token n,
 *   R_t = l R_{t+1} + scale dO_t q_t^T before it,
 *   dk_t = R_t^T v_t,  dv_t = R_t k_t,  dS0 = l R_1 (dS_T where there are no tokens).
 * Nothing is kept from the forward call. dS0 is neither S0 nor dS_T. */
vla_status vla_decay_backward(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO,
                              vla_dtype dtype, int B, int H, int T, int d, const float* log_decay, float scale,
                              const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                              const vla_seq_out* dk, const vla_seq_out* dv, float* dS0, void* scratch,
                              size_t scratch_bytes, void* status, void* stream);

/* Both with options (NULL: the defaults), of which the waits' are read:
 *   wait_limit_us        limit of every in-kernel wait (0: 2,000,000). The bf16
 *                        kernel for more than 8 tokens has such waits
 *   test_stall_producer  TESTING ONLY: nonzero keeps back the last tokens' loads in
 *                        that kernel, so that its waits run out: VLA_ERR_TIMEOUT in
 *                        the status record, role = the block's group of four warps */
vla_status vla_decay_forward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H,
                                int T, int d, const float* log_decay, float scale, const int* lengths,
                                const float* S0, const vla_seq_out* o, float* S_out, void* scratch,
                                size_t scratch_bytes, void* status, void* stream, const vla_options* opts);
vla_status vla_decay_backward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO,
                                 vla_dtype dtype, int B, int H, int T, int d, const float* log_decay, float scale,
                                 const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                                 const vla_seq_out* dk, const vla_seq_out* dv, float* dS0, void* scratch,
                                 size_t scratch_bytes, void* status, void* stream, const vla_options* opts);

/* One token of the recurrence for B sequences, their states updated in place
 * in a pool: q, k, v, o [B, H, d] of dtype, contiguous, 16-byte aligned;
 * states [N, H, d, d] float32, 16-byte aligned. slots: [B] int32 on the
 * device, the pool entry of each sequence, or NULL for entry b (B <= N). A
 * negative slot is an idle row: no state is touched and its o is zero. A slot
 * >= N, and the second and later use of a slot in one call, are treated the
 * same and set VLA_ERR_BAD_SLOT in the status record ({role 4, b, slot}). */
vla_status vla_decay_step(const void* q, const void* k, const void* v, vla_dtype dtype, int B, int H, int d,
                          const float* log_decay, float scale, float* states, int N, const int* slots, void* o,
                          void* status, void* stream);

/* ---- the gated delta rule -----------------------------------------------------
 *
 *   S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   o_t = scale S_t q_t,
 *   a_t = exp(log_decay_t)
 *
 * Each token corrects what the decayed memory gives for its key towards its value:
 * beta 1 and a unit key replace it, beta 0 leaves it. S as above. Keys are taken
 * as they are (vla_qk_norm() makes them unit rows); where beta |k|^2 is above 2 the
 * recurrence itself grows without bound.
 *
 * log_decay and beta are float32 gates for each token and head, at any strides
 * (vla_gate). log_decay NULL: 0. Values below -256 count as -256 (a factor of 0);
 * values above 0 are taken as they are, and a head that grows beyond float32 within
 * 32 tokens gives Inf or NaN. lengths: as for vla_decay_forward().
 *
 * Rounding. fp32 calls, and of bf16 calls the states, dS0 and dbeta: fp32 throughout.
 * bf16 o, dq and dv: rounded at the end, of terms within 2^-14, so that errors are
 * those of rounding the exact result, about 1.65e-3 of a row's size. bf16 dk: the
 * same of dv as it was written, whose rounding meets some of the terms: 1.7e-3 to
 * 2e-3. dlog_decay of a token is the sum of the terms that its decay multiplies where
 * it is below -2 (bf16: -6), about 2e-7 off (bf16: up to 2e-4, by dv); above that a
 * difference of larger sums, off by about 2^-22 of |o.dO| + |v.dv| + |R||S| over its
 * block of 64 tokens (32 in fp32): up to 1e-5 of it (bf16: 1e-4) at the lowest
 * decays, less than 3e-6 at decays above -1. 0 below -256.
 *
 * A token's NaN or Inf reaches the results that depend on it, and may reach those of
 * other tokens of its block of 64 in the same head. One in an output sets VLA_ERR_NONFINITE
 * in the status record; a bounded in-kernel wait that ran out VLA_ERR_TIMEOUT. */

/* Gates [B, H, T] float32: element (b, h, t) is data[b * stride_b + h * stride_h +
 * t * stride_t]. data is 4-byte aligned; the strides of dimensions longer than 1
 * are not negative; 0 repeats a value (else VLA_ERR_INVALID_ARG). */
typedef struct {
    const float* data;
    long long stride_b, stride_h, stride_t;
} vla_gate;

/* The same for an output; the strides are positive. */
typedef struct {
    float* data;
    long long stride_b, stride_h, stride_t;
} vla_gate_out;

/* The rule over T tokens. S0, S_out and T == 0 as for vla_decay_forward(); S_out
 * may be S0. */
vla_status vla_delta_forward(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H, int T,
                             int d, const vla_gate* log_decay, const vla_gate* beta, float scale, const int* lengths,
                             const float* S0, const vla_seq_out* o, float* S_out, void* status, void* stream);

/* Device scratch of vla_delta_backward(), 256-byte aligned, one call's own (0 for
 * sizes that it refuses): the recurrence's corrections, 4 d bytes a token and head;
 * two states every 64 tokens (32 in fp32) and two more a head; 3 d / 4 bytes a token
 * and head for the gates' gradients. */
size_t vla_delta_scratch_bytes(vla_dtype dtype, int B, int H, int T, int d);

/* Reverse mode of vla_delta_forward(): from dO = dL/do and dS_T = dL/dS_out (NULL:
 * zero) the gradients dq, dk, dv, dlog_decay (may be NULL), dbeta and, unless NULL,
 * dS0 = dL/dS0. With R the gradient of S_t (scale dO_t q_t^T and later tokens' part),
 * e_t = v_t - a_t S_{t-1} k_t and D_t = a_t S_{t-1}:
 *   dq_t = scale S_t^T dO_t,  dbeta_t = (R k_t) . e_t,  dv_t = beta_t R k_t,
 *   dk_t = beta_t R^T e_t - D_t^T dv_t,  R' = R - dv_t k_t^T,
 *   dlog_decay_t = <R', D_t>,  and a_t R' is what S_{t-1} gets.
 * Nothing is kept from the forward call. Rows behind a sequence's end are written
 * as zero. dS0 is neither S0 nor dS_T. A gate of stride 0 gets its gradients
 * token by token; their sum is the caller's. */
vla_status vla_delta_backward(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO, vla_dtype dtype,
                              int B, int H, int T, int d, const vla_gate* log_decay, const vla_gate* beta, float scale,
                              const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                              const vla_seq_out* dk, const vla_seq_out* dv, const vla_gate_out* dlog_decay,
                              const vla_gate_out* dbeta, float* dS0, void* scratch, size_t scratch_bytes, void* status,
                              void* stream);

/* Both with options, as vla_decay_forward_ex() and vla_decay_backward_ex(): bf16 calls of
 * more than 64 tokens have in-kernel waits. */
vla_status vla_delta_forward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H, int T,
                                int d, const vla_gate* log_decay, const vla_gate* beta, float scale, const int* lengths,
                                const float* S0, const vla_seq_out* o, float* S_out, void* status, void* stream,
                                const vla_options* opts);
vla_status vla_delta_backward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO, vla_dtype dtype,
                                 int B, int H, int T, int d, const vla_gate* log_decay, const vla_gate* beta, float scale,
                                 const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                                 const vla_seq_out* dk, const vla_seq_out* dv, const vla_gate_out* dlog_decay,
                                 const vla_gate_out* dbeta, float* dS0, void* scratch, size_t scratch_bytes, void* status,
                                 void* stream, const vla_options* opts);

/* One token of the rule for B sequences, their states updated in place in a pool;
 * log_decay (NULL: 0) and beta [B, H] float32, contiguous; the rest as for
 * vla_decay_step(). fp32 throughout. */
vla_status vla_delta_step(const void* q, const void* k, const void* v, vla_dtype dtype, int B, int H, int d,
                          const float* log_decay, const float* beta, float scale, float* states, int N,
                          const int* slots, void* o, void* status, void* stream);

/* ---- norm and position rotation of queries and keys ----------------------------
 *
 * For each row x (the d values of a q or k of one (b, h, t)):
 *   z = x rstd weight[h],  rstd = 1 / sqrt(mean(x^2) + eps), or 1 / sqrt(sum(x^2) + eps)
 * where unit is nonzero (rows of length 1 for a delta rule), and then, with m = rot / 2
 * and the angles a_i = position freqs[i],
 *   y_i = z_i cos a_i - z_(i+m) sin a_i,  y_(i+m) = z_(i+m) cos a_i + z_i sin a_i  (i < m),
 * the coordinates from rot on as they are. rot is a multiple of 16, 0 (none) to d.
 *
 * weight_q, weight_k: float32, 16-byte aligned, [H, d], or [d] where shared is nonzero;
 * NULL: 1. freqs: [rot / 2] float64 on the device, radians a position (not read where
 * rot is 0). positions: int32 on the device, that of token t of sequence b at
 * positions[b * positions_stride_b + t] (stride 0: the same for all), or NULL for t.
 * Angles are as exact as products of float64 values at any position. fp32 throughout; y rounded at
 * the end. rstd_q, rstd_k: [B, H, T] float32, written (NULL: not) by the forward call and
 * read by the backward call. yq may be the rows of q, and yk those of k. */
vla_status vla_qk_norm(const vla_seq* q, const vla_seq* k, vla_dtype dtype, int B, int H, int T, int d,
                       const float* weight_q, const float* weight_k, int shared, int unit, float eps,
                       const double* freqs, int rot, const int* positions, long long positions_stride_b,
                       const vla_seq_out* yq, const vla_seq_out* yk, float* rstd_q, float* rstd_k, void* stream);

/* Bytes of scratch vla_qk_norm_backward() needs for the weights' gradients, on the
 * current device. */
size_t vla_qk_norm_scratch_bytes(int B, int H, int T, int d);

/* Reverse mode: dq, dk of dtype from dyq, dyk and the forward call's q, k and rstd;
 * dweight_q, dweight_k (float32, shaped as the weights; both or neither NULL) are sums
 * over the rows in an order that depends on the sizes and the device alone. dq may be the
 * rows of dyq or q, and dk those of dyk or k. */
vla_status vla_qk_norm_backward(const vla_seq* dyq, const vla_seq* dyk, const vla_seq* q, const vla_seq* k,
                                vla_dtype dtype, int B, int H, int T, int d, const float* weight_q,
                                const float* weight_k, int shared, int unit, const double* freqs, int rot,
                                const int* positions, long long positions_stride_b, const float* rstd_q,
                                const float* rstd_k, const vla_seq_out* dq, const vla_seq_out* dk, float* dweight_q,
                                float* dweight_k, void* scratch, size_t scratch_bytes, void* stream);

/* ---- layer norm of each head's readout --------------------------------------
 *
 *   y = (x - mean) rstd weight[h] + bias[h] over the d values of a row,
 *   rstd = 1 / sqrt(var + eps), var the mean of (x - mean)^2.
 *
 * weight, bias: float32, 16-byte aligned, [H, d], or [d] where shared is
 * nonzero; NULL: 1 and 0. mean, rstd: [B, H, T] float32, written by the
 * forward call (NULL: not written) and read by the backward call. x and y may
 * be the same rows. */
vla_status vla_head_norm(const vla_seq* x, vla_dtype dtype, int B, int H, int T, int d, const float* weight,
                         const float* bias, int shared, float eps, const vla_seq_out* y, float* mean, float* rstd,
                         void* stream);

/* Bytes of scratch vla_head_norm_backward() needs for dweight and dbias. */
size_t vla_head_norm_scratch_bytes(int B, int H, int T, int d);

/* dx [B, H, T, d] of dtype; dweight and dbias (float32, shaped as weight; both
 * or neither NULL) are sums over the rows in an order that depends on the
 * sizes alone. dx may be dy's or x's rows. */
vla_status vla_head_norm_backward(const vla_seq* dy, const vla_seq* x, vla_dtype dtype, int B, int H, int T, int d,
                                  const float* weight, int shared, const float* mean, const float* rstd,
                                  const vla_seq_out* dx, float* dweight, float* dbias, void* scratch,
                                  size_t scratch_bytes, void* stream);

/* ---- quantised cache of states ----------------------------------------------
 *
 * A cache has N slots of `rows` x d values (rows = H * d for a matrix state,
 * H for z^key) in 8 or 4 bits with one float32 scale per 32 values of a row:
 * scale = amax / 127 (bits 8) or amax / 7 (bits 4), code = value / scale
 * rounded to the nearest whole number (ties to even; the quotient is not
 * rounded first), value = code * scale. A group whose scale would be below
 * 2^-126 is stored as zero; one that holds a NaN or Inf is read back as NaN
 * and sets VLA_ERR_NONFINITE.
 *   codes   bits 8: [N, rows, d] int8; bits 4: [N, rows, d / 2] bytes, value
 *           2 i in the low half of byte i. 16-byte aligned.
 *   scales  [N, rows, d / 32] float32
 * (both may be NULL where N is 0). slots as for vla_decay_step(), NULL for slot b. B <= 65535. */

/* Write x [B, rows, d] float32 (16-byte aligned) into slots. A negative slot is skipped; one
 * >= N or used before in the call is skipped and sets VLA_ERR_BAD_SLOT. */
vla_status vla_state_store(const float* x, int B, long long rows, int d, int bits, void* codes, float* scales, int N,
                           const int* slots, void* status, void* stream);

/* Read slots into x [B, rows, d] float32. The same slot may be read more than
 * once. A negative slot reads as zero (a fresh state), and so does one >= N,
 * which also sets VLA_ERR_BAD_SLOT. */
vla_status vla_state_load(const void* codes, const float* scales, int N, const int* slots, int B, long long rows,
                          int d, int bits, float* x, void* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VLA_GB300_LAYER_H */
