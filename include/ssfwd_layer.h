/*
 * ssfwd_layer.h - the part of libssfwd.so's C ABI with the operators of a gated
 * recurrent layer beside its projections:
 *
 *   ss_gated_scan           linear recurrence per channel whose decay and input
 *                           are set by gates, on dense batches
 *   ss_gated_scan_bwd       its backward
 *   ss_packed_gated_scan    the same recurrence over packed requests, with a
 *                           cache of states by slot
 *   ss_gated_state_update   the same for one token per request
 *   ss_rms_norm             root-mean-square norm of a sum with the residual
 *   ss_rms_norm_bwd         its backward
 *   ss_rms_norm_quant       the same norm with an output in e4m3 and scales
 *
 * The pages that the scan operators cite describe neither; formulas stand at each
 * declaration. Conventions are those of ssfwd.h: device pointers owned by the
 * caller, work enqueued on `stream`, nothing allocated, every check before
 * anything is enqueued, strides in elements. Statuses are ss_status. A wait of a kernel
 * of the recurrence (for a copy, or for a CTA of its cluster) gives up after about a
 * second, sets the error word of ss_device_error and runs on.
 */
#ifndef SSFWD_LAYER_H_
#define SSFWD_LAYER_H_

#include "ssfwd_packed.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated linear recurrence. For channel c and token t of a sequence:
 *
 *     r = sigmoid(gate[t,c]),  i = sigmoid(input_gate[t,c])    (1 without it)
 *     L = -rate * softplus(decay[c]) * r,   a = exp(L)
 *     h = a * h + sqrt(1 - a^2) * i * x[t,c],   out[t,c] = h
 *
 * h starts from initial_state (zero when NULL) and is held in fp32; out is h
 * rounded once, last_state the last token's h. What a state loses is 2^-24 of the largest
 * before it per token. decay is finite; a gate may be infinite (open or shut). A NaN, or
 * an infinite state, is a NaN from its next token on, in its channel and sequence alone.
 * The factor sqrt(1 - a^2) is every token's, the first one's too: layers that take it as 1
 * where a document starts are not this one.
 *
 *   x, gate, input_gate, out  (batch, seqlen, dim) in dtype, dim stride 1; stride
 *                {batch, token}. input_gate may be NULL.
 *   decay        (dim,) fp32. rate: finite, > 0.
 *   initial_state, last_state (batch, dim) fp32, contiguous; either may be NULL.
 *   kept         (batch, ceil(seqlen / SS_GATED_TILE), dim) fp32, contiguous, or
 *                NULL: the state before every SS_GATED_TILE-th token, from which
 *                the backward takes up the recurrence.
 *
 *   workspace    ss_gated_scan_workspace_size bytes, 16-byte aligned (0 bytes where
 *                sequences and channels alone fill the device): maps of parts of a
 *                sequence, which run side by side.
 *
 * batch * ceil(dim / 32) < 2^24, 1 <= seqlen (batch may be 0), seqlen and dim < 2^31 -
 * 2^20. out overlaps no input.
 */
#define SS_GATED_TILE 64

typedef struct ss_gated_scan_params {
  int32_t abi_version, dtype;
  float rate;
  int32_t reserved0;
  int64_t batch, seqlen, dim;
  const void *x, *gate, *input_gate;
  const float *decay, *initial_state;
  void *out;
  float *last_state, *kept;
  int64_t x_stride[2], gate_stride[2], input_gate_stride[2], out_stride[2];
  void *workspace;
  int64_t workspace_bytes;
} ss_gated_scan_params;

int ss_gated_scan_validate(const ss_gated_scan_params *p);
int ss_gated_scan_workspace_size(const ss_gated_scan_params *p, int64_t *bytes);
int ss_gated_scan(const ss_gated_scan_params *p, void *stream);

/*
 * Backward, for dout = dL/dout and dlast = dL/dlast_state (zero when NULL), with
 * `kept` as ss_gated_scan left it. Backwards over the tokens, with e past the last
 * one dlast and q = |L| / sqrt(1 - a^2) (0 where L is 0):
 *
 *     g = dout + e,  e = a * g
 *     dx = g sqrt(1 - a^2) i,   dinput_gate = g sqrt(1 - a^2) i (1 - i) x
 *     G = g (a h[t-1] L + i x a^2 q),   dgate = G (1 - r)
 *     ddecay = sum over sequences and tokens of G * sigmoid(decay) / softplus(decay)
 *     dinitial_state = e before the first token
 *
 * An infinite or NaN dout, dlast or state makes gradients of its channel and sequence
 * infinite or NaN, which of the two is not said.
 *
 * dx, dgate, dinput_gate (in dtype), ddecay (dim,) and dinitial_state (batch, dim)
 * fp32 may be NULL (not wanted). workspace: ss_gated_scan_bwd_workspace_size
 * bytes, 16-byte aligned; sums are made in the same order in every call.
 */
typedef struct ss_gated_scan_bwd_params {
  int32_t abi_version, dtype;
  float rate;
  int32_t reserved0;
  int64_t batch, seqlen, dim;
  const void *x, *gate, *input_gate, *dout;
  const float *decay, *kept, *dlast;
  void *dx, *dgate, *dinput_gate;
  float *ddecay, *dinitial_state;
  int64_t x_stride[2], gate_stride[2], input_gate_stride[2], dout_stride[2], dx_stride[2], dgate_stride[2], dinput_gate_stride[2];
  void *workspace;
  int64_t workspace_bytes;
} ss_gated_scan_bwd_params;

int ss_gated_scan_bwd_validate(const ss_gated_scan_bwd_params *p);
int ss_gated_scan_bwd_workspace_size(const ss_gated_scan_bwd_params *p, int64_t *bytes);
int ss_gated_scan_bwd(const ss_gated_scan_bwd_params *p, void *stream);

/*
 * The recurrence over packed requests (tables of ss_request_tables): h of request r
 * starts as state[slot] when context > 0, else 0, and ends in state[slot]. A request
 * without tokens, or with slot -1, leaves the cache alone. Two requests must not
 * share a slot. out is 0 past the last token.
 *
 *   x, gate, input_gate, out  (tokens, dim) in dtype, dim stride 1.
 *   state        (slots, dim) fp32, rows of state_stride; NULL: every request starts
 *                from 0 and nothing is kept.
 *   workspace    ss_packed_gated_scan_workspace_size bytes, 16-byte aligned.
 */
typedef struct ss_packed_gated_scan_params {
  int32_t abi_version, dtype;
  float rate;
  int32_t reserved0;
  int64_t dim, slots;
  const void *x, *gate, *input_gate;
  const float *decay;
  float *state;
  void *out;
  int64_t x_stride, gate_stride, input_gate_stride, out_stride, state_stride;
  ss_packed_tables tables;
  void *workspace;
  int64_t workspace_bytes;
} ss_packed_gated_scan_params;

int ss_packed_gated_scan_validate(const ss_packed_gated_scan_params *p);
int ss_packed_gated_scan_workspace_size(const ss_packed_gated_scan_params *p, int64_t *bytes);
int ss_packed_gated_scan(const ss_packed_gated_scan_params *p, void *stream);

/* One token per request: row r goes with state slot_map[r] (or r, when slot_map
 * is NULL), which is read and written. A row with slot -1 gets out = 0. Two rows
 * must not share a slot. At most 65535 requests. */
typedef struct ss_gated_state_update_params {
  int32_t abi_version, dtype;
  float rate;
  int32_t reserved0;
  int64_t requests, dim, slots;
  const void *x, *gate, *input_gate;
  const float *decay;
  const int32_t *slot_map;
  float *state;
  void *out;
  int64_t x_stride, gate_stride, input_gate_stride, out_stride, state_stride;
} ss_gated_state_update_params;

int ss_gated_state_update_validate(const ss_gated_state_update_params *p);
int ss_gated_state_update(const ss_gated_state_update_params *p, void *stream);

/*
 * Root-mean-square norm of rows, with the residual's addition:
 *
 *     s = x + residual, rounded to residual_dtype      (x itself without a residual)
 *     out = s / sqrt(mean(s^2) + eps) * weight
 *
 * The norm takes s as it is kept, so that the backward, which reads the kept sum,
 * is the gradient of what the forward computed. Squares are summed in fp32: a row whose
 * sum of squares passes its range (values from some 2^64 / sqrt(dim) on) comes out as zeros.
 *
 *   x, out       (rows, dim) in dtype; residual, sum (rows, dim) in residual_dtype,
 *                which is dtype or fp32 and ignored without a residual. dim stride 1.
 *                residual and sum may be NULL; sum needs residual.
 *   weight       (dim,) in weight_dtype, dtype or fp32; contiguous.
 *   rstd         (rows,) fp32, or NULL: 1 / sqrt(mean(s^2) + eps), for the backward.
 *
 * 1 <= dim <= SS_NORM_MAX_DIM, rows < 2^31 - 2^20, eps >= 0. Neither out nor sum
 * overlaps an input, but sum may be residual itself.
 */
#define SS_NORM_MAX_DIM 32768

typedef struct ss_rms_norm_params {
  int32_t abi_version, dtype, residual_dtype, weight_dtype;
  float eps;
  int32_t reserved0;
  int64_t rows, dim;
  const void *x, *residual, *weight;
  void *out, *sum;
  float *rstd;
  int64_t x_stride, residual_stride, out_stride, sum_stride;
} ss_rms_norm_params;

int ss_rms_norm_validate(const ss_rms_norm_params *p);
int ss_rms_norm(const ss_rms_norm_params *p, void *stream);

/*
 * Backward, for dout = dL/dout and dsum = dL/dsum (zero when NULL), with s the sum
 * (or x) and rstd of the forward, n = s rstd and m the mean over the row:
 *
 *     ds = rstd (weight dout - n m(weight dout n)) + dsum
 *     dx = ds, dresidual = ds,   dweight = sum over rows of dout n
 *
 * dout and dx (rows, dim) in dtype; s, dsum and dresidual in residual_dtype. dx,
 * dresidual and dweight (in weight_dtype) may be NULL (not wanted). workspace:
 * ss_rms_norm_bwd_workspace_size bytes, 16-byte aligned; sums are made in the same
 * order in every call.
 */
typedef struct ss_rms_norm_bwd_params {
  int32_t abi_version, dtype, residual_dtype, weight_dtype;
  int64_t rows, dim;
  const void *dout, *dsum, *sum, *weight;
  const float *rstd;
  void *dx, *dresidual, *dweight;
  int64_t dout_stride, dsum_stride, sum_stride, dx_stride, dresidual_stride;
  void *workspace;
  int64_t workspace_bytes;
} ss_rms_norm_bwd_params;

int ss_rms_norm_bwd_validate(const ss_rms_norm_bwd_params *p);
int ss_rms_norm_bwd_workspace_size(const ss_rms_norm_bwd_params *p, int64_t *bytes);
int ss_rms_norm_bwd(const ss_rms_norm_bwd_params *p, void *stream);

/*
 * The norm with an output in e4m3 (finite, no infinities): for each group of
 * `group` channels of a row (0: the whole row; 32, 64 or 128), with v the norm's
 * values in fp32 and most the largest of |v|,
 *
 *     scale = max(most / 448, 2^-126)          (SS_SCALE_F32)
 *     scale = the least power of two not below that   (SS_SCALE_E8M0)
 *     out = v / scale rounded to nearest even, so that v is about out * scale
 *
 * The quotient is v times the scale's reciprocal: exact for a power of two, within 2^-23
 * of it for an fp32 scale, which itself is rounded once. A group with a NaN or an infinity
 * among its v has scale NaN and is NaN throughout. An infinite s makes its own v NaN and
 * the rest of its row zeros.
 *
 *   out          (rows, dim) bytes, dim stride 1.
 *   scale        (rows, ceil(dim / group)) fp32, or bytes of e8m0; contiguous, row by
 *                row: a product that wants scales in tiles reorders them itself.
 */
typedef enum ss_scale_type { SS_SCALE_F32 = 0, SS_SCALE_E8M0 = 1 } ss_scale_type;

typedef struct ss_rms_norm_quant_params {
  int32_t abi_version, dtype, residual_dtype, weight_dtype;
  float eps;
  int32_t scale_type;
  int64_t rows, dim, group;
  const void *x, *residual, *weight;
  void *out, *scale, *sum;
  int64_t x_stride, residual_stride, out_stride, sum_stride;
} ss_rms_norm_quant_params;

int ss_rms_norm_quant_validate(const ss_rms_norm_quant_params *p);
int ss_rms_norm_quant(const ss_rms_norm_quant_params *p, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSFWD_LAYER_H_ */
