// C ABI of the packed operators (include/ssfwd_packed.h): argument checks and
// launches. Every check is made before anything is enqueued.
#include "ssfwd_packed.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "ss_packed.h"

namespace {

int elem_size(int dt) { return dt == SS_F32 ? 4 : 2; }
bool bad_dtype(int dt) { return dt < SS_F32 || dt > SS_BF16; }
bool aligned(const void *p, int a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Host-side fault injection for tests, as in the other entry points:
// SSFWD_FAULT=launch makes the launch report a CUDA failure.
bool launch_fault() {
  const char *f = std::getenv("SSFWD_FAULT");
  return f && std::strcmp(f, "launch") == 0;
}

int launched(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ERR_CUDA; }

struct Range {
  uintptr_t lo, hi;
};
// The bytes of an operand with the given sizes and strides (outermost first).
Range span(const void *ptr, int64_t esize, std::initializer_list<int64_t> sizes, std::initializer_list<int64_t> strides) {
  if (!ptr) return {0, 0};
  int64_t last = 0;
  auto st = strides.begin();
  for (int64_t n : sizes) {
    if (n == 0) return {0, 0};
    last += (n - 1) * *st++;
  }
  const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
  return {lo, lo + static_cast<uintptr_t>((last + 1) * esize)};
}
bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
// Rows interleaved in one buffer (the parts of a projection's output) have
// overlapping spans and no common element: allowed when both have the same row
// stride and their row parts are disjoint within it.
bool rows_meet(Range a, int64_t row_a, Range b, int64_t row_b, int64_t stride_a, int64_t stride_b) {
  if (!overlap(a, b)) return false;
  if (stride_a != stride_b || stride_a <= 0) return true;
  const int64_t d = static_cast<int64_t>((a.lo > b.lo ? a.lo - b.lo : b.lo - a.lo) % stride_a);
  const int64_t lo = a.lo > b.lo ? row_b : row_a, hi = a.lo > b.lo ? row_a : row_b;
  return d < lo || d + hi > stride_a;
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (int64_t(1) << 20);
constexpr int64_t kMaxBlock = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool bad_stride(int64_t s) { return s < 0 || s > kMaxStride; }

int64_t most_blocks(int64_t tokens, int64_t block, int64_t requests) {
  return tokens / block + std::min(requests, tokens);
}

int validate_sizes(int64_t requests, int64_t tokens, int64_t block, int64_t max_blocks) {
  if (requests < 1 || tokens < 0 || block < 1) return SS_ERR_SHAPE;
  if (requests > SS_MAX_REQUESTS || tokens >= kMaxTokens || block >= kMaxBlock) return SS_ERR_UNSUPPORTED;
  if (max_blocks != most_blocks(tokens, block, requests)) return SS_ERR_SHAPE;
  return SS_OK;
}

// ---- request tables ----

int validate(const ss_request_tables_params *p) {
  if (!p) return SS_ERR_NULL;
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  const int st = validate_sizes(p->requests, p->tokens, p->block, p->max_blocks);
  if (st != SS_OK) return st;
  if (p->free < 0) return SS_ERR_SHAPE;
  if (p->free > kMaxTokens) return SS_ERR_UNSUPPORTED;
  if (!p->lengths || !p->offsets || !p->slot_map || !p->counts) return SS_ERR_NULL;
  if (p->tokens > 0 && (!p->token_request || !p->token_position || !p->blocks)) return SS_ERR_NULL;
  if (p->tokens >= p->block && !p->carried) return SS_ERR_NULL;
  for (const void *q : {(const void *)p->lengths, (const void *)p->context, (const void *)p->slots, (const void *)p->free_slots})
    if (q && !aligned(q, 4)) return SS_ERR_ALIGN;
  for (const void *q : {(const void *)p->offsets, (const void *)p->token_request, (const void *)p->token_position,
                        (const void *)p->blocks, (const void *)p->carried, (const void *)p->slot_map, (const void *)p->counts})
    if (!aligned(q, 16)) return SS_ERR_ALIGN;
  const Range ins[4] = {span(p->lengths, 4, {p->requests}, {1}), span(p->context, 4, {p->requests}, {1}),
                        span(p->slots, 4, {p->requests}, {1}), span(p->free_slots, 4, {p->free}, {1})};
  const Range outs[7] = {span(p->offsets, 4, {p->requests + 1}, {1}), span(p->token_request, 4, {p->tokens}, {1}),
                         span(p->token_position, 4, {p->tokens}, {1}), span(p->blocks, 4, {4 * p->max_blocks}, {1}),
                         span(p->slot_map, 4, {p->requests}, {1}), span(p->counts, 4, {4}, {1}),
                         span(p->carried, 4, {p->tokens / p->block}, {1})};
  for (int i = 0; i < 7; ++i) {
    for (const Range &in : ins)
      if (overlap(outs[i], in)) return SS_ERR_ALIAS;
    for (int k = 0; k < i; ++k)
      if (overlap(outs[i], outs[k])) return SS_ERR_ALIAS;
  }
  return SS_OK;
}

// The tables as an operator's input.
int validate(const ss_packed_tables &t) {
  const int st = validate_sizes(t.requests, t.tokens, t.block, t.max_blocks);
  if (st != SS_OK) return st;
  if (t.tokens == 0) return SS_OK;
  if (!t.offsets || !t.token_request || !t.blocks || !t.slot_map || !t.counts) return SS_ERR_NULL;
  if (t.tokens >= t.block && !t.carried) return SS_ERR_NULL;
  for (const void *q : {(const void *)t.offsets, (const void *)t.token_request, (const void *)t.blocks, (const void *)t.carried,
                        (const void *)t.slot_map, (const void *)t.counts})
    if (!aligned(q, 16)) return SS_ERR_ALIGN;
  if (t.context && !aligned(t.context, 4)) return SS_ERR_ALIGN;
  return SS_OK;
}
ssk::Tables tables_of(const ss_packed_tables &t) {
  return {(int)t.requests, (int)t.tokens, (int)t.block, (int)t.max_blocks, t.offsets, t.token_request, t.blocks,
          t.carried, t.slot_map, t.counts, t.context};
}

// ---- packed convolution ----

template <typename P>
int validate_conv(const P *p, int64_t rows) {
  if (bad_dtype(p->dtype)) return SS_ERR_DTYPE;
  if (p->activation != SS_ACT_NONE && p->activation != SS_ACT_SILU) return SS_ERR_UNSUPPORTED;
  if (p->dim < 1 || p->slots < 0) return SS_ERR_SHAPE;
  if (p->width < 2 || p->width > 4 || p->dim > (int64_t(1) << 20) || p->slots > (int64_t(1) << 31)) return SS_ERR_UNSUPPORTED;
  if (rows == 0) return SS_OK;
  if (!p->x || !p->weight || !p->out) return SS_ERR_NULL;
  if (bad_stride(p->x_stride) || bad_stride(p->out_stride) || (p->conv_state && bad_stride(p->state_stride))) return SS_ERR_STRIDE;
  if (p->out_stride < p->dim && rows > 1) return SS_ERR_STRIDE;  // rows of out must not overlap
  const int es = elem_size(p->dtype);
  const int64_t win = p->dim * (p->width - 1);
  if (p->conv_state && p->slots > 1 && p->state_stride < win) return SS_ERR_STRIDE;
  if (!aligned(p->x, es) || !aligned(p->out, es) || !aligned(p->weight, 4) || (p->bias && !aligned(p->bias, 4)) ||
      (p->conv_state && !aligned(p->conv_state, es)))
    return SS_ERR_ALIGN;
  const Range x = span(p->x, es, {rows, p->dim}, {p->x_stride, 1}), out = span(p->out, es, {rows, p->dim}, {p->out_stride, 1});
  const Range st = span(p->conv_state, es, {p->slots, win}, {p->state_stride, 1});
  const Range w = span(p->weight, 4, {p->dim * p->width}, {1}), b = span(p->bias, 4, {p->dim}, {1});
  const int64_t row = p->dim * es;
  if (rows_meet(out, row, x, row, p->out_stride * es, p->x_stride * es) || overlap(out, w) || overlap(out, b) ||
      overlap(out, st) || overlap(st, x) || overlap(st, w) || overlap(st, b))
    return SS_ERR_ALIAS;
  return SS_OK;
}

// 16-byte accesses: every row and window starts on 16 bytes, and holds whole pieces.
template <typename P>
int conv_vec(const P *p, int64_t rows) {
  const int es = elem_size(p->dtype), v = 16 / es;
  return p->dim % v == 0 && aligned(p->x, 16) && aligned(p->out, 16) && (rows == 1 || (p->x_stride % v == 0 && p->out_stride % v == 0)) &&
         (!p->conv_state || (aligned(p->conv_state, 16) && (p->slots <= 1 || p->state_stride % v == 0)));
}

int validate(const ss_packed_conv1d_params *p) {
  if (!p) return SS_ERR_NULL;
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  const int st = validate(p->tables);
  return st != SS_OK ? st : validate_conv(p, p->tables.tokens);
}

int validate(const ss_packed_conv1d_update_params *p) {
  if (!p) return SS_ERR_NULL;
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  if (p->requests < 0) return SS_ERR_SHAPE;
  if (p->requests >= kMaxTokens) return SS_ERR_UNSUPPORTED;
  const int st = validate_conv(p, p->requests);
  if (st != SS_OK || p->requests == 0) return st;
  if (!p->conv_state) return SS_ERR_NULL;
  if (p->slot_map && !aligned(p->slot_map, 4)) return SS_ERR_ALIGN;
  if (!p->slot_map && p->slots < p->requests) return SS_ERR_SHAPE;
  const Range m = span(p->slot_map, 4, {p->requests}, {1});
  const int es = elem_size(p->dtype);
  if (overlap(m, span(p->out, es, {p->requests, p->dim}, {p->out_stride, 1})) ||
      overlap(m, span(p->conv_state, es, {p->slots, p->dim * (p->width - 1)}, {p->state_stride, 1})))
    return SS_ERR_ALIAS;
  return SS_OK;
}

// ---- headed scan ----

template <typename P>
int validate_heads(const P *p, int64_t rows) {
  if (bad_dtype(p->dtype) || (p->dt_dtype != SS_F32 && p->dt_dtype != p->dtype)) return SS_ERR_DTYPE;
  if (p->heads < 1 || p->headdim < 1 || p->dstate < 1 || p->ngroups < 1 || p->heads % p->ngroups != 0 || p->slots < 0)
    return SS_ERR_SHAPE;
  if (p->headdim > 256 || p->dstate > 256 || p->heads > 8192 || p->slots > (int64_t(1) << 31)) return SS_ERR_UNSUPPORTED;
  if (rows == 0) return SS_OK;
  if (!p->x || !p->dt || !p->A || !p->B || !p->C || !p->out) return SS_ERR_NULL;
  for (int i = 0; i < 2; ++i)
    if (bad_stride(p->x_stride[i]) || bad_stride(p->dt_stride[i]) || bad_stride(p->B_stride[i]) || bad_stride(p->C_stride[i]) ||
        (p->z && bad_stride(p->z_stride[i])) || bad_stride(p->out_stride[i]) || (p->state && bad_stride(p->state_stride[i])))
      return SS_ERR_STRIDE;
  // what is written must not overlap itself: heads within a row, rows (or slots) apart
  const int64_t H = p->heads, P_ = p->headdim, N = p->dstate, G = p->ngroups;
  if ((H > 1 && p->out_stride[1] < P_) || (rows > 1 && p->out_stride[0] < (H - 1) * p->out_stride[1] + P_)) return SS_ERR_STRIDE;
  if (p->state && ((H > 1 && p->state_stride[1] < P_ * N) ||
                   (p->slots > 1 && p->state_stride[0] < (H - 1) * p->state_stride[1] + P_ * N)))
    return SS_ERR_STRIDE;
  const int es = elem_size(p->dtype), ds = elem_size(p->dt_dtype);
  const void *rows16[5] = {p->x, p->B, p->C, p->z, p->out};
  for (const void *q : rows16)
    if (q && !aligned(q, es)) return SS_ERR_ALIGN;
  if (!aligned(p->dt, ds)) return SS_ERR_ALIGN;
  const void *words[4] = {p->A, p->D, p->dt_bias, p->state};
  for (const void *q : words)
    if (q && !aligned(q, 4)) return SS_ERR_ALIGN;
  const Range out = span(p->out, es, {rows, H, P_}, {p->out_stride[0], p->out_stride[1], 1});
  const Range st = span(p->state, 4, {p->slots, H, P_ * N}, {p->state_stride[0], p->state_stride[1], 1});
  const int64_t out_row = ((H - 1) * p->out_stride[1] + P_) * es;
  auto meets = [&](const void *ptr, int64_t e, int64_t n, int64_t w, const int64_t *s) {
    const Range r = span(ptr, e, {rows, n, w}, {s[0], s[1], 1});
    return overlap(st, r) || rows_meet(out, out_row, r, ((n - 1) * s[1] + w) * e, p->out_stride[0] * es, s[0] * e);
  };
  if (meets(p->x, es, H, P_, p->x_stride) || meets(p->B, es, G, N, p->B_stride) || meets(p->C, es, G, N, p->C_stride) ||
      (p->z && meets(p->z, es, H, P_, p->z_stride)) || meets(p->dt, ds, H, 1, p->dt_stride) || overlap(out, st))
    return SS_ERR_ALIAS;
  for (int i = 0; i < 3; ++i) {
    const Range r = span(words[i], 4, {H}, {1});
    if (overlap(out, r) || overlap(st, r)) return SS_ERR_ALIAS;
  }
  return SS_OK;
}

// Blocks past a request's first exist only where a request can be longer than one.
bool may_split(const ss_packed_tables &t) { return t.tokens > t.block; }

ssk::HeadScanParams scan_params(const ss_head_scan_params *p) {
  ssk::HeadScanParams k{};
  k.heads = (int)p->heads;
  k.headdim = (int)p->headdim;
  k.dstate = (int)p->dstate;
  k.hpg = (int)(p->heads / p->ngroups);
  k.softplus = p->dt_softplus != 0;
  k.dt_f32 = p->dt_dtype == SS_F32;
  k.split = may_split(p->tables);
  k.slots = p->slots;
  k.x = p->x; k.dt = p->dt; k.B = p->B; k.C = p->C; k.z = p->z;
  k.A = p->A; k.D = p->D; k.bias = p->dt_bias;
  k.state = p->state;
  k.out = p->out;
  for (int i = 0; i < 2; ++i) {
    k.sx[i] = p->x_stride[i]; k.sdt[i] = p->dt_stride[i]; k.sB[i] = p->B_stride[i]; k.sC[i] = p->C_stride[i];
    k.sz[i] = p->z ? p->z_stride[i] : 0; k.so[i] = p->out_stride[i]; k.ss[i] = p->state ? p->state_stride[i] : 0;
  }
  k.vec = p->dstate % 4 == 0 && (!p->state || (aligned(p->state, 16) && (p->heads == 1 || k.ss[1] % 4 == 0) &&
                                               (p->slots <= 1 || k.ss[0] % 4 == 0)));
  k.t = tables_of(p->tables);
  return k;
}

// Workspace: the summaries' states and decays, then copies of the operands that do
// not lie in 16-byte rows, each on 16 bytes.
struct Workspace {
  int64_t states = 0, decays = 0, copies = 0, bytes = 0;  // values; offset of the copies; all
  int64_t rows_x = 0, rows_bc = 0;                        // bytes of one copy of x, z or out; of B or C
  int unaligned = 0;
};
Workspace workspace_of(const ss_head_scan_params *p) {
  Workspace w;
  if (p->tables.tokens == 0) return w;
  if (may_split(p->tables)) {
    w.decays = p->tables.max_blocks * p->heads;
    w.states = w.decays * p->headdim * p->dstate;
  }
  w.copies = w.bytes = (w.states + w.decays) * 4;
  const ssk::HeadScanParams k = scan_params(p);
  if (!ssk::head_scan_tc_sizes(p->dtype, k) || (w.unaligned = ssk::head_scan_tc_unaligned(k)) == 0) return w;
  w.copies = (w.bytes + 15) / 16 * 16;
  w.rows_x = p->tables.tokens * p->heads * ((p->headdim + 7) / 8) * 16;
  w.rows_bc = p->tables.tokens * p->ngroups * ((p->dstate + 7) / 8) * 16;
  const int u = w.unaligned;
  w.bytes = w.copies + w.rows_x * (!!(u & ssk::kRowsX) + !!(u & ssk::kRowsZ) + !!(u & ssk::kRowsOut)) +
            w.rows_bc * (!!(u & ssk::kRowsB) + !!(u & ssk::kRowsC));
  return w;
}

// Whether every launch of the scan is one that a grid holds (its second dimension
// does at all sizes that validate_heads lets through).
bool grids_fit(const ss_head_scan_params *p) {
  constexpr int64_t most = 0x7fffffff;
  const ssk::HeadScanParams k = scan_params(p);
  if (k.split && ssk::head_scan_carry_ctas(k) > most) return false;
  if (!ssk::head_scan_tc_sizes(p->dtype, k)) return true;
  if (ssk::head_scan_tc_tiles(k) * (p->tables.max_blocks + 1) > most) return false;
  const int u = ssk::head_scan_tc_unaligned(k);
  const bool wide = u & (ssk::kRowsX | ssk::kRowsZ | ssk::kRowsOut), narrow = u & (ssk::kRowsB | ssk::kRowsC);
  return !(wide && ssk::copy_rows_ctas(k.t.tokens, k.heads, k.headdim) > most) &&
         !(narrow && ssk::copy_rows_ctas(k.t.tokens, (int)p->ngroups, k.dstate) > most);
}

int validate_operands(const ss_head_scan_params *p) {
  if (!p) return SS_ERR_NULL;
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  int st = validate(p->tables);
  if (st == SS_OK) st = validate_heads(p, p->tables.tokens);
  if (st != SS_OK || p->tables.tokens == 0) return st;
  return grids_fit(p) ? SS_OK : SS_ERR_UNSUPPORTED;
}

int validate(const ss_head_scan_params *p) {
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  const int64_t need = workspace_of(p).bytes;
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return SS_ERR_SCRATCH;
  if (need > 0 && !aligned(p->workspace, 16)) return SS_ERR_ALIGN;
  return SS_OK;
}

int validate(const ss_head_state_update_params *p) {
  if (!p) return SS_ERR_NULL;
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  if (p->requests < 0) return SS_ERR_SHAPE;
  if (p->requests > 65535) return SS_ERR_UNSUPPORTED;
  const int st = validate_heads(p, p->requests);
  if (st != SS_OK || p->requests == 0) return st;
  if (!p->state) return SS_ERR_NULL;
  if (p->slot_map && !aligned(p->slot_map, 4)) return SS_ERR_ALIGN;
  if (!p->slot_map && p->slots < p->requests) return SS_ERR_SHAPE;
  return SS_OK;
}

}  // namespace

extern "C" {

int ss_request_tables_validate(const ss_request_tables_params *p) { return validate(p); }

int ss_request_tables(const ss_request_tables_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (launch_fault()) return SS_ERR_CUDA;
  const ssk::TablesParams k = {(int)p->requests, (int)p->tokens, (int)p->block, (int)p->max_blocks, (int)p->free,
                               p->lengths, p->context, p->slots, p->free_slots, p->offsets, p->token_request,
                               p->token_position, p->blocks, p->carried, p->slot_map, p->counts};
  return launched(ssk::launch_request_tables(k, static_cast<cudaStream_t>(stream)));
}

int ss_packed_conv1d_validate(const ss_packed_conv1d_params *p) { return validate(p); }

int ss_packed_conv1d(const ss_packed_conv1d_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->tables.tokens == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  const ssk::PackedConvParams k = {(int)p->dim, (int)p->width, p->activation, conv_vec(p, p->tables.tokens), p->slots,
                                   p->x_stride, p->out_stride, p->state_stride, p->x, p->weight, p->bias,
                                   p->conv_state, p->out, tables_of(p->tables)};
  return launched(ssk::launch_packed_conv(p->dtype, k, static_cast<cudaStream_t>(stream)));
}

int ss_packed_conv1d_update_validate(const ss_packed_conv1d_update_params *p) { return validate(p); }

int ss_packed_conv1d_update(const ss_packed_conv1d_update_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->requests == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  const ssk::PackedConvUpdateParams k = {(int)p->requests, (int)p->dim, (int)p->width, p->activation, conv_vec(p, p->requests),
                                         p->slots, p->x_stride, p->out_stride, p->state_stride, p->x, p->weight, p->bias,
                                         p->slot_map, p->conv_state, p->out};
  return launched(ssk::launch_packed_conv_update(p->dtype, k, static_cast<cudaStream_t>(stream)));
}

int ss_head_scan_validate(const ss_head_scan_params *p) { return validate(p); }

int ss_head_scan_workspace_size(const ss_head_scan_params *p, int64_t *bytes) {
  if (!bytes) return SS_ERR_NULL;
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  *bytes = workspace_of(p).bytes;
  return SS_OK;
}

int ss_head_scan(const ss_head_scan_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->tables.tokens == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  ssk::HeadScanParams k = scan_params(p);
  const Workspace w = workspace_of(p);
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (k.split) {
    k.ws_state = static_cast<float *>(p->workspace);
    k.ws_decay = k.ws_state + w.states;
  }
  k.err = ssk::packed_error_word();
  if (!k.err) return SS_ERR_CUDA;
  if (!ssk::head_scan_tc_sizes(p->dtype, k)) return launched(ssk::launch_head_scan(p->dtype, k, st_));
  const ssk::TensorMapEncode enc = ssk::packed_map_encode();
  if (!enc) return SS_ERR_CUDA;
  // operands that TMA cannot describe go through rows that it can: a copy of them
  // costs a fraction of what the form without tensor cores takes
  char *at = static_cast<char *>(p->workspace) + w.copies;
  const int tokens = k.t.tokens, groups = (int)p->ngroups;
  cudaError_t e = cudaSuccess;
  auto to_rows = [&](int which, const void *&ptr, long long *strides, int rows, int width, int64_t bytes) {
    if (!(w.unaligned & which) || e != cudaSuccess) return;
    e = ssk::launch_to_rows(ptr, strides, at, tokens, rows, width, st_);
    ptr = at;
    strides[1] = (width + 7) / 8 * 8;
    strides[0] = rows * strides[1];
    at += bytes;
  };
  to_rows(ssk::kRowsX, k.x, k.sx, k.heads, k.headdim, w.rows_x);
  to_rows(ssk::kRowsZ, k.z, k.sz, k.heads, k.headdim, w.rows_x);
  to_rows(ssk::kRowsB, k.B, k.sB, groups, k.dstate, w.rows_bc);
  to_rows(ssk::kRowsC, k.C, k.sC, groups, k.dstate, w.rows_bc);
  if (e != cudaSuccess) return SS_ERR_CUDA;
  void *const out = k.out;
  const long long so[2] = {k.so[0], k.so[1]};
  if (w.unaligned & ssk::kRowsOut) {
    k.out = at;
    k.so[1] = (k.headdim + 7) / 8 * 8;
    k.so[0] = k.heads * k.so[1];
  }
  e = ssk::launch_head_scan_tc(p->dtype, k, enc, st_);
  if (e == cudaSuccess && (w.unaligned & ssk::kRowsOut)) e = ssk::launch_from_rows(k.out, out, so, tokens, k.heads, k.headdim, st_);
  return launched(e);
}

int64_t ss_head_scan_block(int64_t tokens, int64_t requests, int64_t heads, int64_t headdim, int32_t dtype, int32_t sms) {
  if (tokens < 1 || requests < 1 || heads < 1 || headdim < 1 || sms < 1) return 128;
  // Requests of the average length, cut into `cut` blocks each: the waves of CTAs,
  // each of so many steps (of 128 tokens on the tensor cores, else of 16), the
  // summaries of all blocks but the last (a third of a step's work) and two more
  // launches. The weights are estimates; against other blocks (captured graphs, us):
  //   65536 tokens x 32 heads bf16    3456: 339    2688 397, 4736 424, 8192 362
  //   2 x 8192 tokens x 24 heads bf16 1408: 99     1024 136, 2048 126, 8192 299
  //   8 x 2048 tokens x 24 heads bf16 2048: 92     1024 126, 512 133
  //   8 ragged, 4096 x 24 heads fp32   176: 276    128 304, 256 360, 64 312
  //   5 ragged, 777 x 6 heads fp32      16: 22     32 24, 64 35, 1024 95
  const bool tc = dtype != SS_F32 && headdim <= 128;
  const int64_t tiles = tc ? (headdim <= 64 ? (heads + 1) / 2 : heads) : heads * ((headdim + 63) / 64);
  const int64_t resident = tc ? sms : 4 * sms, step = tc ? 128 : 16;
  const int64_t steps = (tokens / requests + step - 1) / step;
  int64_t best = 1;
  double least = 0;
  for (int64_t cut = 1; cut <= std::min<int64_t>(std::max<int64_t>(steps, 1), 64); ++cut) {
    const int64_t len = (steps + cut - 1) / cut;
    const double waves = static_cast<double>((requests * tiles * cut + resident - 1) / resident);
    const double cost = cut > 1 ? waves * (len * 1.34 + 0.5) + 1.5 : waves * len;
    if (cut == 1 || cost < least) {
      least = cost;
      best = cut;
    }
  }
  int64_t block = (steps + best - 1) / best * step;
  // A batch whose requests need no cut may still hold one long request (40 ragged
  // requests, 6001 tokens x 16 heads fp16, rule 1024: 46 us; 512 57, 256 58).
  if (best == 1) block = std::max(block, (tc ? 8 : 4) * step);
  return std::min<int64_t>(std::max<int64_t>(block, step), 1 << 19);
}

int ss_head_state_update_validate(const ss_head_state_update_params *p) { return validate(p); }

int ss_head_state_update(const ss_head_state_update_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->requests == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  ssk::HeadUpdateParams k{};
  k.requests = (int)p->requests;
  k.heads = (int)p->heads;
  k.headdim = (int)p->headdim;
  k.dstate = (int)p->dstate;
  k.hpg = (int)(p->heads / p->ngroups);
  k.softplus = p->dt_softplus != 0;
  k.dt_f32 = p->dt_dtype == SS_F32;
  k.slots = p->slots;
  k.x = p->x; k.dt = p->dt; k.B = p->B; k.C = p->C; k.z = p->z;
  k.A = p->A; k.D = p->D; k.bias = p->dt_bias;
  k.slot_map = p->slot_map;
  k.state = p->state;
  k.out = p->out;
  for (int i = 0; i < 2; ++i) {
    k.sx[i] = p->x_stride[i]; k.sdt[i] = p->dt_stride[i]; k.sB[i] = p->B_stride[i]; k.sC[i] = p->C_stride[i];
    k.sz[i] = p->z ? p->z_stride[i] : 0; k.so[i] = p->out_stride[i]; k.ss[i] = p->state_stride[i];
  }
  k.vec = p->dstate % 4 == 0 && aligned(p->state, 16) && (p->heads == 1 || p->state_stride[1] % 4 == 0) &&
          (p->slots <= 1 || p->state_stride[0] % 4 == 0);
  const int need = 4 * elem_size(p->dtype);
  auto rows_ok = [&](const void *base, const int64_t *s) {
    return aligned(base, need) && (p->requests == 1 || s[0] % 4 == 0) && (p->ngroups == 1 || s[1] % 4 == 0);
  };
  k.bcvec = rows_ok(p->B, p->B_stride) && rows_ok(p->C, p->C_stride);
  return launched(ssk::launch_head_update(p->dtype, k, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
