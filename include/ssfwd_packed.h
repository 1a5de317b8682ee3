/*
 * ssfwd_packed.h - the part of libssfwd.so's C ABI that serves packed requests:
 * one batch of requests of different lengths, their tokens one after another in
 * (tokens, channels) operands without padding, each request with a slot in a
 * cache of states. Five operators:
 *
 *   ss_request_tables       offsets, token maps, block table and slot map from
 *                           the request lengths, on the GPU
 *   ss_packed_conv1d        short causal depthwise convolution of the packed
 *                           tokens, with a cache of windows by slot
 *   ss_packed_conv1d_update the same for one token per request
 *   ss_head_scan            selective scan with one decay per head over the
 *                           packed tokens, with a cache of states by slot
 *   ss_head_state_update    the same for one token per request
 *
 * The pages that the other operators cite describe the scan with a decay per
 * (channel, state), on a dense (batch, dim, seqlen) batch; the operators here
 * have no counterpart on them. Formulas stand at each declaration.
 *
 * Conventions are those of ssfwd.h: device pointers owned by the caller, work
 * enqueued on `stream`, nothing allocated, every check before anything is
 * enqueued, strides in elements. Statuses are ss_status.
 */
#ifndef SSFWD_PACKED_H_
#define SSFWD_PACKED_H_

#include "ssfwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Tables of a packed batch of `requests` requests, of which request r brings
 * lengths[r] >= 0 tokens (an empty request is allowed) and has had context[r]
 * tokens before (context NULL: none has).
 *
 *   offsets[r]         first token of request r; offsets[requests] = all tokens
 *   token_request[t]   the request of token t; -1 past the last token
 *   token_position[t]  context[r] + t - offsets[r]; 0 past the last token
 *   blocks[i]          {request, first token, tokens, index in the request} of
 *                      the i-th run of at most `block` tokens of one request;
 *                      {-1, 0, 0, 0} past the last
 *   carried[i]         the i-th row of blocks that is not its request's last
 *                      (tokens / block of them at most); -1 past the last
 *   slot_map[r]        slots[r] where it is >= 0, else free_slots[k] for the
 *                      k-th such request in order, else (free_slots used up or
 *                      NULL) -1; with slots NULL, r itself
 *   counts             {tokens, blocks, slots taken from free_slots, errors};
 *                      errors is a sum of 1: lengths exceed `tokens` (requests
 *                      are cut there), 2: a negative length (taken as 0),
 *                      4: free_slots used up
 *
 * All tables are contiguous int32, 16-byte aligned; the outputs overlap no
 * input. Sizes: 1 <= requests <= SS_MAX_REQUESTS, 0 <= tokens < 2^31 - 2^20,
 * 1 <= block < 2^20, max_blocks = tokens / block + min(requests, tokens), free
 * >= 0.
 */
#define SS_MAX_REQUESTS 16384

typedef struct ss_request_tables_params {
  int32_t abi_version, reserved0;
  int64_t requests, tokens, block, max_blocks, free;
  const int32_t *lengths, *context, *slots, *free_slots;
  int32_t *offsets, *token_request, *token_position, *blocks, *carried, *slot_map, *counts;
} ss_request_tables_params;

int ss_request_tables_validate(const ss_request_tables_params *p);
int ss_request_tables(const ss_request_tables_params *p, void *stream);

/* The tables as the packed operators read them (outputs of ss_request_tables,
 * and the context it was given, or NULL). */
typedef struct ss_packed_tables {
  int64_t requests, tokens, block, max_blocks;
  const int32_t *offsets, *token_request, *blocks, *carried, *slot_map, *counts, *context;
} ss_packed_tables;

/*
 * Causal depthwise convolution of packed tokens, width W:
 *
 *     out[t,c] = act(bias[c] + sum_{k<W} weight[c,k] * x[t-(W-1)+k, c])
 *
 * where the tokens before the first of t's request are its slot's window
 * (conv_state[slot, c, :], oldest first) when context > 0, else 0. Afterwards
 * the window holds the request's last W-1 inputs. A request without tokens, or
 * with slot -1, leaves the cache alone. Two requests must not share a slot. out
 * is 0 past the last token.
 *
 *   x, out       (tokens, dim) in dtype, dim stride 1.
 *   weight       (dim, width) fp32, contiguous; 2 <= width <= 4, dim <= 2^20.
 *   bias         (dim,) fp32, or NULL.
 *   conv_state   (slots, dim, width-1) in dtype, contiguous but for its slot
 *                stride; NULL: every request starts from 0 and nothing is kept.
 */
typedef struct ss_packed_conv1d_params {
  int32_t abi_version, dtype, activation, reserved0;
  int64_t dim, width, slots;
  const void *x;
  const float *weight, *bias;
  void *conv_state, *out;
  int64_t x_stride, out_stride, state_stride;
  ss_packed_tables tables;
} ss_packed_conv1d_params;

int ss_packed_conv1d_validate(const ss_packed_conv1d_params *p);
int ss_packed_conv1d(const ss_packed_conv1d_params *p, void *stream);

/* One token per request: row r of x goes with window slot_map[r] (or r, when
 * slot_map is NULL). A row with slot -1 gets out = 0. Two rows must not share
 * a slot. */
typedef struct ss_packed_conv1d_update_params {
  int32_t abi_version, dtype, activation, reserved0;
  int64_t requests, dim, width, slots;
  const void *x;
  const float *weight, *bias;
  const int32_t *slot_map;
  void *conv_state, *out;
  int64_t x_stride, out_stride, state_stride;
} ss_packed_conv1d_update_params;

int ss_packed_conv1d_update_validate(const ss_packed_conv1d_update_params *p);
int ss_packed_conv1d_update(const ss_packed_conv1d_update_params *p, void *stream);

/*
 * Selective scan with one decay per head. For request r, head h of group
 * g = h / (heads / ngroups), and its state S (headdim x dstate), token by token:
 *
 *     dt      = softplus(dt[t,h] + dt_bias[h])        (plain sum if !dt_softplus)
 *     S[p,n]  = exp(dt * A[h]) * S[p,n] + dt * x[t,h,p] * B[t,g,n]
 *     y[p]    = sum_n C[t,g,n] * S[p,n] + D[h] * x[t,h,p]
 *     out     = y * silu(z[t,h,p]) if z is given, else y
 *
 * S starts as state[slot, h] when context > 0, else 0, and ends in
 * state[slot, h]. A request without tokens, or with slot -1, leaves the cache
 * alone. Two requests must not share a slot. out is 0 past the last token.
 *
 *   x, z, out    (tokens, heads, headdim) in dtype, last stride 1; stride
 *                {token, head}. z may be NULL.
 *   dt           (tokens, heads), dtype or fp32 (dt_dtype); stride {token, head}.
 *   B, C         (tokens, ngroups, dstate) in dtype, last stride 1.
 *   A, D, dt_bias (heads,) fp32; D and dt_bias may be NULL (0).
 *   state        (slots, heads, headdim, dstate) fp32, stride {slot, head},
 *                the last two contiguous; NULL: every request starts from 0
 *                and nothing is kept.
 *   workspace    ss_head_scan_workspace_size bytes, 16-byte aligned; needed
 *                when a request may have more than one block (tokens > block),
 *                and for 16-bit operands that do not lie in rows of 16 bytes.
 *
 * Sizes: 1 <= headdim, dstate <= 256, heads <= 8192 and a multiple of ngroups;
 * tokens / block x heads x ceil(headdim x dstate / 1024) and, on the tensor cores,
 * (max_blocks + 1) x tiles (of two heads of a group, or one above 64) < 2^31.
 *
 * A may have either sign; negative A is what decays.
 *
 * 16-bit operands with headdim, dstate <= 128 run on the tensor cores, 128
 * tokens at a time; the state stays in fp32. Its sums take every bit of bf16
 * operands. A term dt x B of fp16 operands is off by at most 2^-22 of itself, or
 * by 2^-24 of the largest weight (dt times the decay to the end) of its 128
 * tokens, or of its block where the request has several; where that weight is
 * below 1e-19 it counts as 0. Two things follow from
 * that form: a NaN or infinity in a token's x also reaches the outputs of the
 * same request's tokens before it in its 128 (never another request's), and the
 * state, and the product of C.B, the decay between two tokens and the earlier
 * one's dt, are rounded to the operands' type where they enter the output, which
 * adds about as much as the output's own rounding (the state that is kept has
 * none of it). In fp16 these have to stay below 65504, and below 6e-5 they keep
 * an absolute 3e-8. Other operands run token by token in fp32.
 */
typedef struct ss_head_scan_params {
  int32_t abi_version, dtype, dt_dtype, dt_softplus;
  int64_t heads, headdim, dstate, ngroups, slots;
  const void *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias;
  float *state;
  void *out;
  int64_t x_stride[2], dt_stride[2], B_stride[2], C_stride[2], z_stride[2], out_stride[2], state_stride[2];
  void *workspace;
  int64_t workspace_bytes;
  ss_packed_tables tables;
} ss_head_scan_params;

int ss_head_scan_validate(const ss_head_scan_params *p);
int ss_head_scan_workspace_size(const ss_head_scan_params *p, int64_t *bytes);
int ss_head_scan(const ss_head_scan_params *p, void *stream);

/* The block (tokens per unit of parallel work) that suits ss_head_scan on a
 * device of `sms` multiprocessors, for ss_request_tables. */
int64_t ss_head_scan_block(int64_t tokens, int64_t requests, int64_t heads, int64_t headdim, int32_t dtype, int32_t sms);

/* One token per request: row r goes with state slot_map[r] (or r, when slot_map
 * is NULL), which is read and written. A row with slot -1 gets out = 0. Two
 * rows must not share a slot. */
typedef struct ss_head_state_update_params {
  int32_t abi_version, dtype, dt_dtype, dt_softplus;
  int64_t requests, heads, headdim, dstate, ngroups, slots;
  const void *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias;
  const int32_t *slot_map;
  float *state;
  void *out;
  int64_t x_stride[2], dt_stride[2], B_stride[2], C_stride[2], z_stride[2], out_stride[2], state_stride[2];
} ss_head_state_update_params;

int ss_head_state_update_validate(const ss_head_state_update_params *p);
int ss_head_state_update(const ss_head_state_update_params *p, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSFWD_PACKED_H_ */
