// C ABI of the layer operators (include/ssfwd_layer.h): argument checks and
// launches. Every check is made before anything is enqueued.
#include "ssfwd_layer.h"

#include <cuda_runtime.h>

#include <cmath>

#include "ss_checks.h"
#include "ss_layer.h"

namespace {

constexpr int64_t kMaxUnits = int64_t(1) << 24;  // (sequence, channel tile) pairs: times a cluster's CTAs or segments a grid holds them

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Makes the current device's context current: a thread's first call (autograd runs
// backward passes on threads of its own) finds none, and the tensor-map encoder wants one.
bool context_ready() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

// A (outer, rows, width) operand whose last stride is 1.
struct Rows {
  const void *ptr;
  int es;
  int64_t outer, rows, width;
  int64_t stride[2];
  bool written;
};
Range span_of(const Rows &r) { return span(r.ptr, r.es, {r.outer, r.rows, r.width}, {r.stride[0], r.stride[1], 1}); }

// Strides, alignment, and that nothing that is written meets anything else. `flat`:
// contiguous buffers, the first `written` of them outputs.
int check_rows(std::initializer_list<Rows> all) {
  for (const Rows &r : all) {
    if (!r.ptr) continue;
    if (bad_stride(r.stride[0]) || bad_stride(r.stride[1])) return SS_ERR_STRIDE;
    if (!aligned(r.ptr, r.es)) return SS_ERR_ALIGN;
    if (r.written && ((r.rows > 1 && r.stride[1] < r.width) ||
                      (r.outer > 1 && r.stride[0] < (r.rows - 1) * r.stride[1] + r.width &&
                       !(r.stride[1] >= r.outer * r.stride[0] && r.stride[0] >= r.width))))
      return SS_ERR_STRIDE;
  }
  for (const Rows *a = all.begin(); a != all.end(); ++a)
    for (const Rows *b = all.begin(); b != all.end(); ++b) {
      if (a == b || !a->ptr || !b->ptr || !a->written || (b->written && b < a)) continue;
      // parts of one row do not meet
      if (a->outer == 1 && b->outer == 1) {
        if (rows_meet(span_of(*a), a->width * a->es, span_of(*b), b->width * b->es, a->stride[1] * a->es, b->stride[1] * b->es)) return SS_ERR_ALIAS;
      } else if (overlap(span_of(*a), span_of(*b))) {
        // parts of one row, in sequences that follow one another at the same distance
        const bool same = a->es == b->es && a->stride[0] == b->stride[0] && a->stride[1] == b->stride[1];
        if (!same || rows_meet(span_of(*a), a->width * a->es, span_of(*b), b->width * b->es, a->stride[1] * a->es, b->stride[1] * b->es) ||
            a->stride[0] < (a->rows - 1) * a->stride[1] + std::max(a->width, b->width) || a->stride[0] % std::max<int64_t>(a->stride[1], 1) != 0)
          return SS_ERR_ALIAS;
      }
    }
  return SS_OK;
}
// Two neighbouring channels of 2 or 4 bytes in one access.
bool pairs(std::initializer_list<Rows> all, int64_t dim) {
  if (dim % 2) return false;
  for (const Rows &r : all)
    if (r.ptr && (!aligned(r.ptr, 2 * r.es) || (r.rows > 1 && r.stride[1] % 2) || (r.outer > 1 && r.stride[0] % 2))) return false;
  return true;
}
// How the recurrence's rows come and go: by TMA where every row is whole pieces of 16
// bytes (a store writes the last one to its end, whatever of it is the row's) and ends
// before the next (rows that are broadcast or windows of one buffer do not: a tensor
// map's strides are those of whole rows), else in pairs or single values.
int rows_kind(std::initializer_list<Rows> all, int64_t dim) {
  auto off = [](int64_t bytes, int64_t row) { return bytes < row || bytes % 16 || bytes >> 40; };
  bool tma = true;
  for (const Rows &r : all)
    if (r.ptr && (!aligned(r.ptr, 16) || r.width * r.es % 16 || (r.rows > 1 && off(r.stride[1] * r.es, r.width * r.es)) ||
                  (r.outer > 1 && off(r.stride[0] * r.es, r.width * r.es))))
      tma = false;
  return tma ? 2 : pairs(all, dim) ? 1 : 0;
}
// 16-byte accesses.
bool sixteens(std::initializer_list<Rows> all, int64_t dim, int v) {
  if (dim % v) return false;
  for (const Rows &r : all)
    if (r.ptr && (!aligned(r.ptr, std::min(16, v * r.es)) || (r.rows > 1 && r.stride[1] * r.es % std::min(16, v * r.es)))) return false;
  return true;
}
bool meets_flat(std::initializer_list<Rows> all, Range flat, bool written) {
  for (const Rows &r : all)
    if (r.ptr && (written || r.written) && overlap(span_of(r), flat)) return true;
  return false;
}

int check_gated(int abi, int dtype, float rate, int64_t dim) {
  if (abi != SS_ABI_VERSION) return SS_ERR_VERSION;
  if (bad_dtype(dtype)) return SS_ERR_DTYPE;
  if (dim < 1) return SS_ERR_SHAPE;
  if (dim >= kMaxTokens || !(rate > 0.f) || !std::isfinite(rate)) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

// ---- gated recurrence ----

#define SS_ROWS3(q, ptr, st, w) Rows{ptr, es, (q)->batch, (q)->seqlen, (q)->dim, {(st)[0], (st)[1]}, w}

int check_dense(int abi, int dtype, float rate, int64_t batch, int64_t seqlen, int64_t dim) {
  const int st = check_gated(abi, dtype, rate, dim);
  if (st != SS_OK) return st;
  if (batch < 0 || seqlen < 0) return SS_ERR_SHAPE;
  if (seqlen >= kMaxTokens || batch >= kMaxUnits || batch * up(dim, ssk::kGatedCh) >= kMaxUnits) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int validate_operands(const ss_gated_scan_params *p) {
  if (!p) return SS_ERR_NULL;
  int st = check_dense(p->abi_version, p->dtype, p->rate, p->batch, p->seqlen, p->dim);
  if (st != SS_OK || p->batch == 0) return st;
  if (p->seqlen == 0) return SS_ERR_SHAPE;
  if (!p->x || !p->gate || !p->decay || !p->out) return SS_ERR_NULL;
  const int es = elem_size(p->dtype);
  const Rows x = SS_ROWS3(p, p->x, p->x_stride, false), g = SS_ROWS3(p, p->gate, p->gate_stride, false),
             i = SS_ROWS3(p, p->input_gate, p->input_gate_stride, false), o = SS_ROWS3(p, p->out, p->out_stride, true);
  st = check_rows({x, g, i, o});
  if (st != SS_OK) return st;
  const int64_t states = p->batch * p->dim;
  const Range flats[4] = {span(p->last_state, 4, {states}, {1}), span(p->kept, 4, {states * up(p->seqlen, SS_GATED_TILE)}, {1}),
                          span(p->decay, 4, {p->dim}, {1}), span(p->initial_state, 4, {states}, {1})};
  for (const void *q : {(const void *)p->last_state, (const void *)p->kept, (const void *)p->decay, (const void *)p->initial_state})
    if (!aligned(q, 4)) return SS_ERR_ALIGN;
  for (int k = 0; k < 4; ++k) {
    if (meets_flat({x, g, i, o}, flats[k], k < 2)) return SS_ERR_ALIAS;
    for (int l = k + 1; l < 4; ++l)
      if (k < 2 && overlap(flats[k], flats[l])) return SS_ERR_ALIAS;
  }
  return SS_OK;
}

int validate_operands(const ss_gated_scan_bwd_params *p) {
  if (!p) return SS_ERR_NULL;
  int st = check_dense(p->abi_version, p->dtype, p->rate, p->batch, p->seqlen, p->dim);
  if (st != SS_OK || p->batch == 0) return st;
  if (p->seqlen == 0) return SS_ERR_SHAPE;
  if (!p->x || !p->gate || !p->decay || !p->dout || !p->kept) return SS_ERR_NULL;
  if (p->dinput_gate && !p->input_gate) return SS_ERR_NULL;
  const int es = elem_size(p->dtype);
  const Rows r[7] = {SS_ROWS3(p, p->x, p->x_stride, false), SS_ROWS3(p, p->gate, p->gate_stride, false),
                     SS_ROWS3(p, p->input_gate, p->input_gate_stride, false), SS_ROWS3(p, p->dout, p->dout_stride, false),
                     SS_ROWS3(p, p->dx, p->dx_stride, true), SS_ROWS3(p, p->dgate, p->dgate_stride, true),
                     SS_ROWS3(p, p->dinput_gate, p->dinput_gate_stride, true)};
  st = check_rows({r[0], r[1], r[2], r[3], r[4], r[5], r[6]});
  if (st != SS_OK) return st;
  const int64_t states = p->batch * p->dim;
  const void *ptrs[5] = {p->ddecay, p->dinitial_state, p->decay, p->dlast, p->kept};
  const int64_t n[5] = {p->dim, states, p->dim, states, states * up(p->seqlen, SS_GATED_TILE)};
  for (int k = 0; k < 5; ++k) {
    if (!aligned(ptrs[k], 4)) return SS_ERR_ALIGN;
    if (meets_flat({r[0], r[1], r[2], r[3], r[4], r[5], r[6]}, span(ptrs[k], 4, {n[k]}, {1}), k < 2)) return SS_ERR_ALIAS;
    for (int l = k + 1; l < 5; ++l)
      if (k < 2 && overlap(span(ptrs[k], 4, {n[k]}, {1}), span(ptrs[l], 4, {n[l]}, {1}))) return SS_ERR_ALIAS;
  }
  return SS_OK;
}
// How the units are shared out, and the workspace for it: the segments' maps, and for the
// backward the parts of ddecay by sequence and CTA.
template <typename P>
ssk::GatedPlan dense_plan(const P *p) {
  return ssk::gated_plan(p->dtype, p->batch * up(p->dim, ssk::kGatedCh), (int)up(p->seqlen, ssk::kGatedTile));
}
int64_t workspace_of(const ss_gated_scan_params *p) {
  return ssk::gated_map_bytes(p->batch * up(p->dim, ssk::kGatedCh), dense_plan(p));
}
int64_t workspace_of(const ss_gated_scan_bwd_params *p) {
  if (p->batch == 0) return 0;
  const ssk::GatedPlan plan = dense_plan(p);
  return ssk::gated_map_bytes(p->batch * up(p->dim, ssk::kGatedCh), plan) + (p->ddecay ? 4 * p->batch * plan.cluster * plan.segs * p->dim : 0);
}
template <typename P>
int check_workspace(const P *p, int64_t need) {
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return SS_ERR_SCRATCH;
  return need > 0 && !aligned(p->workspace, 16) ? SS_ERR_ALIGN : SS_OK;
}
int validate(const ss_gated_scan_params *p) {
  const int st = validate_operands(p);
  return st != SS_OK ? st : check_workspace(p, workspace_of(p));
}
int validate(const ss_gated_scan_bwd_params *p) {
  const int st = validate_operands(p);
  return st != SS_OK ? st : check_workspace(p, workspace_of(p));
}

#define SS_ROWS2(n, ptr, st, w) Rows{ptr, es, 1, n, p->dim, {0, st}, w}

// The operands that the packed recurrence and its step share.
template <typename P>
int check_by_slot(const P *p, int64_t rows, const int32_t *slot_map) {
  if (p->slots < 0) return SS_ERR_SHAPE;
  if (p->slots > (int64_t(1) << 31)) return SS_ERR_UNSUPPORTED;
  if (rows == 0) return SS_OK;
  if (!p->x || !p->gate || !p->decay || !p->out) return SS_ERR_NULL;
  const int es = elem_size(p->dtype);
  const Rows x = SS_ROWS2(rows, p->x, p->x_stride, false), g = SS_ROWS2(rows, p->gate, p->gate_stride, false),
             i = SS_ROWS2(rows, p->input_gate, p->input_gate_stride, false), o = SS_ROWS2(rows, p->out, p->out_stride, true);
  const Rows st{p->state, 4, 1, p->slots, p->dim, {0, p->state_stride}, true};
  const int status = check_rows({x, g, i, o});
  if (status != SS_OK) return status;
  if (p->state) {
    if (bad_stride(p->state_stride) || (p->slots > 1 && p->state_stride < p->dim)) return SS_ERR_STRIDE;
    if (!aligned(p->state, 4)) return SS_ERR_ALIGN;
    if (meets_flat({x, g, i, o}, span_of(st), true)) return SS_ERR_ALIAS;
  }
  if (!aligned(p->decay, 4) || !aligned(slot_map, 4)) return SS_ERR_ALIGN;
  for (const Range f : {span(p->decay, 4, {p->dim}, {1}), span(slot_map, 4, {rows}, {1})})
    if (overlap(f, span_of(o)) || (p->state && overlap(f, span_of(st)))) return SS_ERR_ALIAS;
  return SS_OK;
}

int validate_operands(const ss_packed_gated_scan_params *p) {
  if (!p) return SS_ERR_NULL;
  int st = check_gated(p->abi_version, p->dtype, p->rate, p->dim);
  if (st == SS_OK) st = validate(p->tables);
  if (st != SS_OK) return st;
  if (up(p->dim, ssk::kGatedCh) >= kMaxUnits) return SS_ERR_UNSUPPORTED;
  return check_by_slot(p, p->tables.tokens, nullptr);
}
ssk::GatedPlan packed_plan(const ss_packed_gated_scan_params *p) {
  return ssk::gated_plan(p->dtype, up(p->dim, ssk::kGatedCh), (int)up(p->tables.tokens, ssk::kGatedTile));
}
int64_t workspace_of(const ss_packed_gated_scan_params *p) { return ssk::gated_map_bytes(up(p->dim, ssk::kGatedCh), packed_plan(p)); }
int validate(const ss_packed_gated_scan_params *p) {
  const int st = validate_operands(p);
  return st != SS_OK ? st : check_workspace(p, workspace_of(p));
}

int validate(const ss_gated_state_update_params *p) {
  if (!p) return SS_ERR_NULL;
  int st = check_gated(p->abi_version, p->dtype, p->rate, p->dim);
  if (st != SS_OK) return st;
  if (p->requests < 0) return SS_ERR_SHAPE;
  if (p->requests > 65535) return SS_ERR_UNSUPPORTED;
  st = check_by_slot(p, p->requests, p->slot_map);
  if (st != SS_OK || p->requests == 0) return st;
  if (!p->state) return SS_ERR_NULL;
  if (!p->slot_map && p->slots < p->requests) return SS_ERR_SHAPE;
  return SS_OK;
}

// ---- norm ----

template <typename P>
int check_norm(const P *p, bool residual) {
  if (p->abi_version != SS_ABI_VERSION) return SS_ERR_VERSION;
  if (bad_dtype(p->dtype) || (p->weight_dtype != SS_F32 && p->weight_dtype != p->dtype) ||
      (residual && p->residual_dtype != SS_F32 && p->residual_dtype != p->dtype))
    return SS_ERR_DTYPE;
  if (p->rows < 0 || p->dim < 1) return SS_ERR_SHAPE;
  if (p->rows >= kMaxTokens || p->dim > SS_NORM_MAX_DIM) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}
template <typename P>
int check_norm_rows(const P *p, int out_es, std::initializer_list<Range> outs) {
  if (!p->x || !p->weight || !p->out || (p->sum && !p->residual)) return SS_ERR_NULL;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return SS_ERR_UNSUPPORTED;
  const int es = elem_size(p->dtype), rs = elem_size(p->residual_dtype), ws = elem_size(p->weight_dtype);
  const Rows x{p->x, es, 1, p->rows, p->dim, {0, p->x_stride}, false};
  const Rows r{p->sum && p->sum == p->residual && p->sum_stride == p->residual_stride ? nullptr : p->residual, rs, 1, p->rows, p->dim, {0, p->residual_stride}, false};
  const Rows o{p->out, out_es, 1, p->rows, p->dim, {0, p->out_stride}, true}, s{p->sum, rs, 1, p->rows, p->dim, {0, p->sum_stride}, true};
  const int st = check_rows({x, r, o, s});
  if (st != SS_OK) return st;
  if (!aligned(p->weight, ws)) return SS_ERR_ALIGN;
  const Range w = span(p->weight, ws, {p->dim}, {1});
  if (meets_flat({x, r, o, s}, w, false)) return SS_ERR_ALIAS;
  for (const Range &f : outs)
    if (meets_flat({x, r, o, s}, f, true) || overlap(f, w)) return SS_ERR_ALIAS;
  return SS_OK;
}

int validate(const ss_rms_norm_params *p) {
  if (!p) return SS_ERR_NULL;
  const int st = check_norm(p, p->residual != nullptr);
  if (st != SS_OK || p->rows == 0) return st;
  if (!aligned(p->rstd, 4)) return SS_ERR_ALIGN;
  return check_norm_rows(p, elem_size(p->dtype), {span(p->rstd, 4, {p->rows}, {1})});
}

int64_t scale_groups(const ss_rms_norm_quant_params *p) { return p->group > 0 ? up(p->dim, p->group) : 1; }

int validate(const ss_rms_norm_quant_params *p) {
  if (!p) return SS_ERR_NULL;
  const int st = check_norm(p, p->residual != nullptr);
  if (st != SS_OK) return st;
  if (p->scale_type != SS_SCALE_F32 && p->scale_type != SS_SCALE_E8M0) return SS_ERR_UNSUPPORTED;
  if (p->group != 0 && p->group != 32 && p->group != 64 && p->group != 128) return SS_ERR_UNSUPPORTED;
  if (p->rows == 0) return SS_OK;
  if (!p->scale) return SS_ERR_NULL;
  const int ss = p->scale_type == SS_SCALE_F32 ? 4 : 1;
  if (!aligned(p->scale, ss)) return SS_ERR_ALIGN;
  return check_norm_rows(p, 1, {span(p->scale, ss, {p->rows * scale_groups(p)}, {1})});
}

int validate_operands(const ss_rms_norm_bwd_params *p) {
  if (!p) return SS_ERR_NULL;
  int st = check_norm(p, true);
  if (st != SS_OK || p->rows == 0) return st;
  if (!p->dout || !p->sum || !p->weight || !p->rstd) return SS_ERR_NULL;
  const int es = elem_size(p->dtype), rs = elem_size(p->residual_dtype), ws = elem_size(p->weight_dtype);
  const int64_t n = p->rows, d = p->dim;
  const Rows r[5] = {{p->dout, es, 1, n, d, {0, p->dout_stride}, false}, {p->dsum, rs, 1, n, d, {0, p->dsum_stride}, false},
                     {p->sum, rs, 1, n, d, {0, p->sum_stride}, false}, {p->dx, es, 1, n, d, {0, p->dx_stride}, true},
                     {p->dresidual, rs, 1, n, d, {0, p->dresidual_stride}, true}};
  st = check_rows({r[0], r[1], r[2], r[3], r[4]});
  if (st != SS_OK) return st;
  if (!aligned(p->weight, ws) || !aligned(p->dweight, ws) || !aligned(p->rstd, 4)) return SS_ERR_ALIGN;
  const Range w = span(p->weight, ws, {d}, {1}), dw = span(p->dweight, ws, {d}, {1}), rstd = span(p->rstd, 4, {n}, {1});
  if (meets_flat({r[0], r[1], r[2], r[3], r[4]}, w, false) || meets_flat({r[0], r[1], r[2], r[3], r[4]}, rstd, false) ||
      meets_flat({r[0], r[1], r[2], r[3], r[4]}, dw, true) || overlap(dw, w) || overlap(dw, rstd))
    return SS_ERR_ALIAS;
  return SS_OK;
}
// Parts of dweight by CTA.
int64_t bwd_workspace(const ss_rms_norm_bwd_params *p) {
  return p->dweight && p->rows > 0 ? 4 * p->dim * ssk::norm_bwd_ctas(p->rows, (int)p->dim) : 0;
}
int validate(const ss_rms_norm_bwd_params *p) {
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  const int64_t need = bwd_workspace(p);
  if (need > 0 && (!p->workspace || p->workspace_bytes < need)) return SS_ERR_SCRATCH;
  if (need > 0 && !aligned(p->workspace, 16)) return SS_ERR_ALIGN;
  return SS_OK;
}

template <typename P>
ssk::NormParams norm_params(const P *p) {
  ssk::NormParams k{};
  k.rows = p->rows;
  k.dim = (int)p->dim;
  k.weight_f32 = p->weight_dtype == SS_F32;
  k.eps = p->eps;
  k.x = p->x; k.residual = p->residual; k.weight = p->weight;
  k.out = p->out; k.sum = p->sum;
  k.sx = p->x_stride; k.sr = p->residual_stride; k.so = p->out_stride; k.ss = p->sum_stride;
  return k;
}
template <typename P>
bool norm_vec(const P *p, int out_es) {
  const int es = elem_size(p->dtype), rs = elem_size(p->residual_dtype), v = es == 4 ? 4 : 8;
  return aligned(p->weight, 16) &&
         sixteens({{p->x, es, 1, p->rows, p->dim, {0, p->x_stride}, false}, {p->residual, rs, 1, p->rows, p->dim, {0, p->residual_stride}, false},
                   {p->out, out_es, 1, p->rows, p->dim, {0, p->out_stride}, true}, {p->sum, rs, 1, p->rows, p->dim, {0, p->sum_stride}, true}},
                  p->dim, v);
}

}  // namespace

extern "C" {

int ss_gated_scan_validate(const ss_gated_scan_params *p) { return validate(p); }

int ss_gated_scan_workspace_size(const ss_gated_scan_params *p, int64_t *bytes) {
  if (!bytes) return SS_ERR_NULL;
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  *bytes = p->batch == 0 ? 0 : workspace_of(p);
  return SS_OK;
}

int ss_gated_scan(const ss_gated_scan_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->batch == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  const bool ready = context_ready();
  const ssk::TensorMapEncode enc = ssk::packed_map_encode();
  ssk::GatedScanParams k{};
  k.err = ssk::packed_error_word();
  if (!ready || !enc || !k.err) return SS_ERR_CUDA;
  k.tokens = (int)p->seqlen;
  k.dim = (int)p->dim;
  k.batch = (int)p->batch;
  k.channel_tiles = (int)up(p->dim, ssk::kGatedCh);
  k.tiles = (int)up(p->seqlen, ssk::kGatedTile);
  k.rate = p->rate;
  k.x = p->x; k.gate = p->gate; k.igate = p->input_gate;
  k.decay = p->decay; k.init = p->initial_state;
  k.out = p->out; k.last = p->last_state; k.kept = p->kept;
  k.plan = dense_plan(p);
  k.maps = p->workspace;
  for (int i = 0; i < 2; ++i) {
    k.sx[i] = p->x_stride[i]; k.sg[i] = p->gate_stride[i]; k.si[i] = p->input_gate_stride[i]; k.so[i] = p->out_stride[i];
  }
  const int es = elem_size(p->dtype);
  const int rows = rows_kind({SS_ROWS3(p, p->x, p->x_stride, false), SS_ROWS3(p, p->gate, p->gate_stride, false),
                           SS_ROWS3(p, p->input_gate, p->input_gate_stride, false), SS_ROWS3(p, p->out, p->out_stride, true)}, p->dim);
  return launched(ssk::launch_gated_scan(p->dtype, rows, enc, k, static_cast<cudaStream_t>(stream)));
}

int ss_gated_scan_bwd_validate(const ss_gated_scan_bwd_params *p) { return validate(p); }

int ss_gated_scan_bwd_workspace_size(const ss_gated_scan_bwd_params *p, int64_t *bytes) {
  if (!bytes) return SS_ERR_NULL;
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  *bytes = workspace_of(p);
  return SS_OK;
}

int ss_gated_scan_bwd(const ss_gated_scan_bwd_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (launch_fault()) return SS_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->batch == 0) return p->ddecay ? launched(cudaMemsetAsync(p->ddecay, 0, 4 * p->dim, s)) : SS_OK;
  const bool ready = context_ready();
  const ssk::TensorMapEncode enc = ssk::packed_map_encode();
  ssk::GatedBwdParams k{};
  k.err = ssk::packed_error_word();
  if (!ready || !enc || !k.err) return SS_ERR_CUDA;
  k.tokens = (int)p->seqlen;
  k.dim = (int)p->dim;
  k.batch = (int)p->batch;
  k.channel_tiles = (int)up(p->dim, ssk::kGatedCh);
  k.tiles = (int)up(p->seqlen, ssk::kGatedTile);
  k.rate = p->rate;
  k.x = p->x; k.gate = p->gate; k.igate = p->input_gate; k.dout = p->dout;
  k.decay = p->decay; k.kept = p->kept; k.dlast = p->dlast;
  k.dx = p->dx; k.dgate = p->dgate; k.digate = p->dinput_gate;
  k.ddecay = p->ddecay; k.dinit = p->dinitial_state;
  k.plan = dense_plan(p);
  k.maps = p->workspace;
  k.parts = p->ddecay ? reinterpret_cast<float *>(static_cast<char *>(p->workspace) + ssk::gated_map_bytes((long long)k.batch * k.channel_tiles, k.plan)) : nullptr;
  for (int i = 0; i < 2; ++i) {
    k.sx[i] = p->x_stride[i]; k.sg[i] = p->gate_stride[i]; k.si[i] = p->input_gate_stride[i]; k.sd[i] = p->dout_stride[i];
    k.sdx[i] = p->dx_stride[i]; k.sdg[i] = p->dgate_stride[i]; k.sdi[i] = p->dinput_gate_stride[i];
  }
  const int es = elem_size(p->dtype);
  const int rows = rows_kind({SS_ROWS3(p, p->x, p->x_stride, false), SS_ROWS3(p, p->gate, p->gate_stride, false),
                           SS_ROWS3(p, p->input_gate, p->input_gate_stride, false), SS_ROWS3(p, p->dout, p->dout_stride, false),
                           SS_ROWS3(p, p->dx, p->dx_stride, true), SS_ROWS3(p, p->dgate, p->dgate_stride, true),
                           SS_ROWS3(p, p->dinput_gate, p->dinput_gate_stride, true)}, p->dim);
  return launched(ssk::launch_gated_bwd(p->dtype, rows, enc, k, s));
}

int ss_packed_gated_scan_validate(const ss_packed_gated_scan_params *p) { return validate(p); }

int ss_packed_gated_scan_workspace_size(const ss_packed_gated_scan_params *p, int64_t *bytes) {
  if (!bytes) return SS_ERR_NULL;
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  *bytes = workspace_of(p);
  return SS_OK;
}

int ss_packed_gated_scan(const ss_packed_gated_scan_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  const int64_t tokens = p->tables.tokens;
  if (tokens == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  const bool ready = context_ready();
  const ssk::TensorMapEncode enc = ssk::packed_map_encode();
  ssk::GatedScanParams k{};
  k.err = ssk::packed_error_word();
  if (!ready || !enc || !k.err) return SS_ERR_CUDA;
  k.tokens = (int)tokens;
  k.dim = (int)p->dim;
  k.batch = 1;
  k.channel_tiles = (int)up(p->dim, ssk::kGatedCh);
  k.tiles = (int)up(tokens, ssk::kGatedTile);
  k.rate = p->rate;
  k.x = p->x; k.gate = p->gate; k.igate = p->input_gate;
  k.decay = p->decay;
  k.out = p->out;
  k.sx[1] = p->x_stride; k.sg[1] = p->gate_stride; k.si[1] = p->input_gate_stride; k.so[1] = p->out_stride;
  k.plan = packed_plan(p);
  k.maps = p->workspace;
  k.token_request = p->tables.token_request;
  k.offsets = p->tables.offsets;
  k.slot_map = p->tables.slot_map;
  k.context = p->tables.context;
  k.state = p->state;
  k.slots = p->slots;
  k.state_stride = p->state_stride;
  const int es = elem_size(p->dtype);
  const int rows = rows_kind({SS_ROWS2(tokens, p->x, p->x_stride, false), SS_ROWS2(tokens, p->gate, p->gate_stride, false),
                           SS_ROWS2(tokens, p->input_gate, p->input_gate_stride, false), SS_ROWS2(tokens, p->out, p->out_stride, true)}, p->dim);
  return launched(ssk::launch_gated_scan(p->dtype, rows, enc, k, static_cast<cudaStream_t>(stream)));
}

int ss_gated_state_update_validate(const ss_gated_state_update_params *p) { return validate(p); }

int ss_gated_state_update(const ss_gated_state_update_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->requests == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  ssk::GatedUpdateParams k{};
  k.rows = (int)p->requests;
  k.dim = (int)p->dim;
  k.rate = p->rate;
  k.slots = p->slots;
  k.x = p->x; k.gate = p->gate; k.igate = p->input_gate;
  k.decay = p->decay;
  k.slot_map = p->slot_map;
  k.state = p->state;
  k.out = p->out;
  k.sx = p->x_stride; k.sg = p->gate_stride; k.si = p->input_gate_stride; k.so = p->out_stride; k.ss = p->state_stride;
  const int es = elem_size(p->dtype);
  const int64_t n = p->requests;
  k.vec = sixteens({SS_ROWS2(n, p->x, p->x_stride, false), SS_ROWS2(n, p->gate, p->gate_stride, false),
                    SS_ROWS2(n, p->input_gate, p->input_gate_stride, false), SS_ROWS2(n, p->out, p->out_stride, true),
                    Rows{p->state, 4, 1, p->slots, p->dim, {0, p->state_stride}, true}}, p->dim, 4);
  return launched(ssk::launch_gated_update(p->dtype, k, static_cast<cudaStream_t>(stream)));
}

int ss_rms_norm_validate(const ss_rms_norm_params *p) { return validate(p); }

int ss_rms_norm(const ss_rms_norm_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->rows == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  ssk::NormParams k = norm_params(p);
  k.rstd = p->rstd;
  return launched(ssk::launch_rms_norm(p->dtype, p->residual_dtype, norm_vec(p, elem_size(p->dtype)), k, static_cast<cudaStream_t>(stream)));
}

int ss_rms_norm_bwd_validate(const ss_rms_norm_bwd_params *p) { return validate(p); }

int ss_rms_norm_bwd_workspace_size(const ss_rms_norm_bwd_params *p, int64_t *bytes) {
  if (!bytes) return SS_ERR_NULL;
  const int st = validate_operands(p);
  if (st != SS_OK) return st;
  *bytes = bwd_workspace(p);
  return SS_OK;
}

int ss_rms_norm_bwd(const ss_rms_norm_bwd_params *p, void *stream) {
  int st = validate(p);
  if (st != SS_OK) return st;
  if (launch_fault()) return SS_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->rows == 0) return p->dweight ? launched(cudaMemsetAsync(p->dweight, 0, elem_size(p->weight_dtype) * p->dim, s)) : SS_OK;
  ssk::NormBwdParams k{};
  k.rows = p->rows;
  k.dim = (int)p->dim;
  k.weight_f32 = p->weight_dtype == SS_F32;
  k.dout = p->dout; k.dsum = p->dsum; k.sum = p->sum; k.weight = p->weight;
  k.rstd = p->rstd;
  k.dx = p->dx; k.dresidual = p->dresidual; k.dweight = p->dweight;
  k.parts = p->dweight ? static_cast<float *>(p->workspace) : nullptr;
  k.ctas = ssk::norm_bwd_ctas(p->rows, k.dim);
  k.sd = p->dout_stride; k.sds = p->dsum_stride; k.ss = p->sum_stride; k.sdx = p->dx_stride; k.sdr = p->dresidual_stride;
  const int es = elem_size(p->dtype), rs = elem_size(p->residual_dtype), v = es == 4 ? 4 : 8;
  const int64_t n = p->rows, d = p->dim;
  const bool vec = aligned(p->weight, 16) && sixteens({{p->dout, es, 1, n, d, {0, p->dout_stride}, false}, {p->dsum, rs, 1, n, d, {0, p->dsum_stride}, false},
                                                       {p->sum, rs, 1, n, d, {0, p->sum_stride}, false}, {p->dx, es, 1, n, d, {0, p->dx_stride}, true},
                                                       {p->dresidual, rs, 1, n, d, {0, p->dresidual_stride}, true}}, d, v);
  return launched(ssk::launch_rms_norm_bwd(p->dtype, p->residual_dtype, vec, k, s));
}

int ss_rms_norm_quant_validate(const ss_rms_norm_quant_params *p) { return validate(p); }

int ss_rms_norm_quant(const ss_rms_norm_quant_params *p, void *stream) {
  const int st = validate(p);
  if (st != SS_OK) return st;
  if (p->rows == 0) return SS_OK;
  if (launch_fault()) return SS_ERR_CUDA;
  ssk::NormParams k = norm_params(p);
  k.group = (int)p->group;
  k.e8m0 = p->scale_type == SS_SCALE_E8M0;
  k.scale = p->scale;
  k.groups = (int)scale_groups(p);
  return launched(ssk::launch_rms_norm_quant(p->dtype, p->residual_dtype, norm_vec(p, 1), k, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
