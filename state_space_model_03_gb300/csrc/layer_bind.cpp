// Python binding of the layer operators (include/ssfwd_layer.h): argument checks,
// output allocation and the call, in C++ for the reason given in packed_bind.cpp.
// init() takes the addresses of libssfwd.so's entry points.
#include "bind_common.h"

#include <ATen/ops/zeros.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>

#include <array>
#include <optional>

#include "ssfwd_layer.h"

namespace {

int (*g_scan)(const ss_gated_scan_params *, void *);
int (*g_scan_ws)(const ss_gated_scan_params *, int64_t *);
int (*g_packed_ws)(const ss_packed_gated_scan_params *, int64_t *);
int (*g_scan_bwd)(const ss_gated_scan_bwd_params *, void *);
int (*g_scan_bwd_ws)(const ss_gated_scan_bwd_params *, int64_t *);
int (*g_packed)(const ss_packed_gated_scan_params *, void *);
int (*g_update)(const ss_gated_state_update_params *, void *);
int (*g_norm)(const ss_rms_norm_params *, void *);
int (*g_norm_bwd)(const ss_rms_norm_bwd_params *, void *);
int (*g_norm_bwd_ws)(const ss_rms_norm_bwd_params *, int64_t *);
int (*g_quant)(const ss_rms_norm_quant_params *, void *);

PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    auto at_ = [&](int i) { return reinterpret_cast<void *>(integer(a[i])); };
    g_scan = reinterpret_cast<decltype(g_scan)>(at_(0));
    g_scan_bwd = reinterpret_cast<decltype(g_scan_bwd)>(at_(1));
    g_scan_bwd_ws = reinterpret_cast<decltype(g_scan_bwd_ws)>(at_(2));
    g_packed = reinterpret_cast<decltype(g_packed)>(at_(3));
    g_update = reinterpret_cast<decltype(g_update)>(at_(4));
    g_norm = reinterpret_cast<decltype(g_norm)>(at_(5));
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(at_(6));
    g_norm_bwd_ws = reinterpret_cast<decltype(g_norm_bwd_ws)>(at_(7));
    g_quant = reinterpret_cast<decltype(g_quant)>(at_(8));
    g_scan_ws = reinterpret_cast<decltype(g_scan_ws)>(at_(9));
    g_packed_ws = reinterpret_cast<decltype(g_packed_ws)>(at_(10));
    g_text = reinterpret_cast<decltype(g_text)>(at_(11));
    Py_INCREF(a[12]);
    g_error = a[12];
    Py_RETURN_NONE;
  });
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
void no_tangent(std::initializer_list<const at::Tensor *> ts) {
  for (const at::Tensor *t : ts)
    if (t && t->_fw_grad(0).defined()) refuse(PyExc_NotImplementedError, "the layer operators take no forward-mode tangents");
}
at::Tensor workspace(int64_t bytes, const at::Tensor &x) {
  return bytes > 0 ? at::empty({bytes}, x.options().dtype(at::kByte)) : at::Tensor();
}
PyObject *wrapped(const at::Tensor &t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject *r = PyTuple_New(ts.size());
  if (!r) throw python_error();
  int i = 0;
  for (const at::Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrapped(t));
  return r;
}
const at::Tensor *f32_of(const at::Tensor *t, const char *name, at::IntArrayRef sizes, const at::Tensor &x) {
  if (t && (t->scalar_type() != at::kFloat || t->sizes() != sizes)) {
    std::string s;
    for (int64_t n : sizes) s += (s.empty() ? "" : ", ") + std::to_string(n);
    refuse(PyExc_TypeError, std::string(name) + " must be float32 (" + s + ")");
  }
  on(t, x, name);
  return t;
}

// x, gate, decay and input_gate, which the three forms of the recurrence share.
struct Gated {
  Held x, gate, igate, decay;
};
template <typename P>
Gated gated_operands(P &p, const at::Tensor &x, const at::Tensor &gate, const at::Tensor &decay, const at::Tensor *igate, float rate,
                     int64_t dims, const char *form) {
  const int dt = dtype_of(x);
  if (x.dim() != dims || dt < 0) refuse(PyExc_TypeError, std::string("x must be ") + form + " fp32/fp16/bf16");
  if (gate.sizes() != x.sizes() || gate.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "gate must match x in shape and dtype");
  if (igate && (igate->sizes() != x.sizes() || igate->scalar_type() != x.scalar_type()))
    refuse(PyExc_TypeError, "input_gate must match x in shape and dtype");
  on(&gate, x, "gate");
  on(igate, x, "input_gate");
  f32_of(&decay, "decay", {x.size(-1)}, x);
  Gated g{rows(&x), rows(&gate), rows(igate), flat(&decay)};
  p.abi_version = SS_ABI_VERSION;
  p.dtype = dt;
  p.rate = rate;
  p.dim = x.size(-1);
  p.x = ptr(g.x.get());
  p.gate = ptr(g.gate.get());
  p.input_gate = ptr(g.igate.get());
  p.decay = fptr(g.decay.get());
  return g;
}
template <int N>
void strides(int64_t (&to)[N], const at::Tensor &t) {
  for (int i = 0; i < N; ++i) to[i] = t.stride(i);
}
template <typename P>
void dense_strides(P &p, const Gated &g) {
  p.batch = g.x.t.size(0);
  p.seqlen = g.x.t.size(1);
  strides(p.x_stride, g.x.t);
  strides(p.gate_stride, g.gate.t);
  if (g.igate.get()) strides(p.input_gate_stride, g.igate.t);
}

void *place(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
const at::Tensor *some(const std::optional<at::Tensor> &t) { return t && t->defined() ? &*t : nullptr; }
std::optional<at::Tensor> maybe(const at::Tensor *t) { return t ? std::optional<at::Tensor>(*t) : std::nullopt; }

struct Scanned {
  at::Tensor out, last, kept;
};
Scanned scan_forward(const at::Tensor &x, const at::Tensor &gate, const at::Tensor &decay, const at::Tensor *igate, float rate,
                     const at::Tensor *init, bool want_last, bool want_kept) {
  ss_gated_scan_params p{};
  const Gated g = gated_operands(p, x, gate, decay, igate, rate, 3, "(batch, seqlen, dim)");
  const Held start = flat(f32_of(init, "initial_state", {x.size(0), x.size(2)}, x));
  dense_strides(p, g);
  const c10::cuda::CUDAGuard guard(x.device());
  Scanned r;
  r.out = at::empty(x.sizes(), x.options());
  const auto f32 = x.options().dtype(at::kFloat);
  if (want_last) r.last = at::empty({p.batch, p.dim}, f32);
  if (want_kept) r.kept = at::empty({p.batch, (p.seqlen + SS_GATED_TILE - 1) / SS_GATED_TILE, p.dim}, f32);
  p.initial_state = fptr(start.get());
  p.out = place(r.out);
  p.last_state = static_cast<float *>(place(r.last));
  p.kept = static_cast<float *>(place(r.kept));
  strides(p.out_stride, r.out);
  check(g_scan_ws(&p, &p.workspace_bytes));
  const at::Tensor ws = workspace(p.workspace_bytes, x);
  p.workspace = place(ws);
  check(g_scan(&p, stream_of(x)));
  return r;
}

enum { kDx, kDgate, kDinput, kDdecay, kDinit, kScanGrads };
// The gradients that `wanted` has a bit for.
std::array<at::Tensor, kScanGrads> scan_backward(const at::Tensor &dout, const at::Tensor *dlast, const at::Tensor &x, const at::Tensor &gate,
                                                 const at::Tensor &decay, const at::Tensor *igate, float rate, const at::Tensor &kept, int wanted) {
  ss_gated_scan_bwd_params p{};
  const Gated g = gated_operands(p, x, gate, decay, igate, rate, 3, "(batch, seqlen, dim)");
  if (dout.sizes() != x.sizes() || dout.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "dout must match x in shape and dtype");
  on(&dout, x, "dout");
  dense_strides(p, g);
  const Held d = rows(&dout), last = flat(f32_of(dlast, "dlast", {p.batch, p.dim}, x));
  f32_of(&kept, "kept", {p.batch, (p.seqlen + SS_GATED_TILE - 1) / SS_GATED_TILE, p.dim}, x);
  const Held starts = flat(&kept);
  const c10::cuda::CUDAGuard guard(x.device());
  const auto f32 = x.options().dtype(at::kFloat);
  std::array<at::Tensor, kScanGrads> r;
  auto wants = [&](int bit) { return (wanted >> bit & 1) != 0; };
  if (wants(kDx)) r[kDx] = at::empty(x.sizes(), x.options());
  if (wants(kDgate)) r[kDgate] = at::empty(x.sizes(), x.options());
  if (wants(kDinput) && igate) r[kDinput] = at::empty(x.sizes(), x.options());
  if (wants(kDdecay)) r[kDdecay] = at::empty({p.dim}, f32);
  if (wants(kDinit)) r[kDinit] = at::empty({p.batch, p.dim}, f32);
  p.dout = d.t.data_ptr();
  strides(p.dout_stride, d.t);
  p.kept = fptr(starts.get());
  p.dlast = fptr(last.get());
  p.dx = place(r[kDx]);
  p.dgate = place(r[kDgate]);
  p.dinput_gate = place(r[kDinput]);
  p.ddecay = static_cast<float *>(place(r[kDdecay]));
  p.dinitial_state = static_cast<float *>(place(r[kDinit]));
  for (int64_t *s : {p.dx_stride, p.dgate_stride, p.dinput_gate_stride}) {
    s[0] = p.seqlen * p.dim;
    s[1] = p.dim;
  }
  check(g_scan_bwd_ws(&p, &p.workspace_bytes));
  const at::Tensor ws = workspace(p.workspace_bytes, x);
  p.workspace = place(ws);
  check(g_scan_bwd(&p, stream_of(x)));
  return r;
}

// A backward pass runs on the engine's threads: what fails there becomes an error that
// the engine hands to the caller.
template <typename F>
auto on_engine(const char *what, F f) {
  try {
    return f();
  } catch (const Refusal &r) {
    TORCH_CHECK(false, what, ": ", r.what);
  } catch (const Status &s) {
    TORCH_CHECK(false, what, ": libssfwd call failed: status ", s.code, " (", g_text(s.code), ")");
  }
}
// Gradients that can be asked for but not differentiated again.
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
variable_list once(const char *what, variable_list grads) {
  if (!c10::GradMode::is_enabled()) return grads;
  for (at::Tensor &t : grads)
    if (t.defined()) t = t.detach().set_requires_grad(true);
  auto refusal = std::make_shared<torch::autograd::DelayedError>(std::string(what) + " is differentiable once", static_cast<int64_t>(grads.size()));
  return (*refusal)(std::move(grads));
}

// gated_scan_fn with its backward: the forward keeps the state before every
// SS_GATED_TILE-th token, from which the backward takes up the recurrence.
struct GatedScan : torch::autograd::Function<GatedScan> {
  static variable_list forward(AutogradContext *ctx, const at::Tensor &x, const at::Tensor &gate, const at::Tensor &decay,
                               const std::optional<at::Tensor> &igate, const std::optional<at::Tensor> &init, double rate, bool want_last) {
    const Scanned r = scan_forward(x, gate, decay, some(igate), static_cast<float>(rate), some(init), want_last, true);
    ctx->save_for_backward({x, gate, decay, igate ? *igate : at::Tensor(), r.kept});
    ctx->saved_data["rate"] = rate;
    ctx->saved_data["init"] = some(init) != nullptr;
    ctx->set_materialize_grads(false);
    return want_last ? variable_list{r.out, r.last} : variable_list{r.out};
  }
  static variable_list backward(AutogradContext *ctx, variable_list d) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &x = saved[0], &igate = saved[3];
    variable_list grads(7);
    const bool last = d.size() > 1 && d[1].defined();
    if (!d[0].defined() && !last) return grads;
    // which gradients are asked for goes by the tensors that were given
    int wanted = 0, edge = 0;
    for (int bit : {kDx, kDgate, kDdecay}) wanted |= ctx->needs_input_grad(edge++) << bit;
    if (igate.defined()) wanted |= ctx->needs_input_grad(edge++) << kDinput;
    if (ctx->saved_data["init"].toBool()) wanted |= ctx->needs_input_grad(edge++) << kDinit;
    std::array<at::Tensor, kScanGrads> r = on_engine("gated_scan_fn's backward", [&] {
      const at::AutoGradMode off(false);
      const at::Tensor dout = d[0].defined() ? d[0] : at::zeros(x.sizes(), x.options());
      return scan_backward(dout, last ? &d[1] : nullptr, x, saved[1], saved[2], igate.defined() ? &igate : nullptr,
                           static_cast<float>(ctx->saved_data["rate"].toDouble()), saved[4], wanted);
    });
    return once("gated_scan_fn", {r[kDx], r[kDgate], r[kDdecay], r[kDinput], r[kDinit], at::Tensor(), at::Tensor()});
  }
};
bool wants_grad(std::initializer_list<const at::Tensor *> ts) {
  if (!c10::GradMode::is_enabled()) return false;
  for (const at::Tensor *t : ts)
    if (t && t->requires_grad()) return true;
  return false;
}

// gated_scan(x, gate, decay, input_gate, rate, initial_state, want_last) -> out or (out, last_state)
PyObject *gated_scan(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 7, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), &gate = need(a[1], "gate"), &decay = need(a[2], "decay"), *igate = opt(a[3], "input_gate");
    const at::Tensor *init = opt(a[5], "initial_state");
    const double rate = number(a[4]);
    const bool want_last = flag(a[6]);
    no_tangent({&x, &gate, &decay, igate, init});
    at::Tensor out, last;
    if (wants_grad({&x, &gate, &decay, igate, init})) {
      const variable_list r = GatedScan::apply(x, gate, decay, maybe(igate), maybe(init), rate, want_last);
      out = r[0];
      if (want_last) last = r[1];
    } else {
      const Scanned r = scan_forward(x, gate, decay, igate, static_cast<float>(rate), init, want_last, false);
      out = r.out;
      last = r.last;
    }
    return want_last ? tuple_of({out, last}) : THPVariable_Wrap(out);
  });
}

// The cache of states (slots, dim) and the rows' strides.
template <typename P>
void by_slot(P &p, const Gated &g, const at::Tensor *state, const at::Tensor &x) {
  if (state) {
    if (state->scalar_type() != at::kFloat || state->dim() != 2 || state->size(1) != p.dim)
      refuse(PyExc_TypeError, "state must be float32 (slots, dim)");
    if (state->numel() && p.dim > 1 && state->stride(1) != 1)
      refuse(PyExc_ValueError, "state must have contiguous rows (it is updated in place)");
    on(state, x, "state");
    p.slots = state->size(0);
    p.state = static_cast<float *>(state->data_ptr());
    p.state_stride = state->stride(0);
  }
  p.x_stride = g.x.t.stride(0);
  p.gate_stride = g.gate.t.stride(0);
  p.input_gate_stride = g.igate.get() ? g.igate.t.stride(0) : 0;
  p.out_stride = p.dim;
}

// packed_gated_scan(x, gate, decay, plan, input_gate, rate, state) -> out
PyObject *packed_gated_scan(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 7, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), &gate = need(a[1], "gate"), &decay = need(a[2], "decay"), *igate = opt(a[4], "input_gate"),
                     *state = opt(a[6], "state");
    ss_packed_gated_scan_params p{};
    const Gated g = gated_operands(p, x, gate, decay, igate, static_cast<float>(number(a[5])), 2, "(tokens, dim)");
    by_slot(p, g, state, x);
    no_grad({&x, &gate, &decay, igate, state});
    p.tables = plan_of(a[3], x).t;
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options());
    p.out = out.data_ptr();
    check(g_packed_ws(&p, &p.workspace_bytes));
    const at::Tensor ws = workspace(p.workspace_bytes, x);
    p.workspace = place(ws);
    check(g_packed(&p, stream_of(x)));
    changed(state);
    return THPVariable_Wrap(std::move(out));
  });
}

// gated_state_update(state, x, gate, decay, input_gate, rate, slots) -> out
PyObject *gated_state_update(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 7, [&]() -> PyObject * {
    const at::Tensor &state = need(a[0], "state"), &x = need(a[1], "x"), &gate = need(a[2], "gate"), &decay = need(a[3], "decay"),
                     *igate = opt(a[4], "input_gate");
    ss_gated_state_update_params p{};
    const Gated g = gated_operands(p, x, gate, decay, igate, static_cast<float>(number(a[5])), 2, "(requests, dim)");
    by_slot(p, g, &state, x);
    no_grad({&x, &gate, &decay, igate, &state});
    p.requests = x.size(0);
    const Held slots = int32(opt(a[6], "slots"), "slots", x.size(0), x);
    p.slot_map = iptr(slots.get());
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options());
    p.out = out.data_ptr();
    check(g_update(&p, stream_of(x)));
    changed(&state);
    return THPVariable_Wrap(std::move(out));
  });
}

// ---- norm ----

// (rows, dim) of a tensor of any number of dimensions, its rows at one distance: without
// a copy where they are so already, as parts of wider rows are.
Held rows2(const at::Tensor *t) {
  if (!t) return Held{};
  const int64_t dim = t->size(-1);
  const at::Tensor r = t->dim() == 2 ? *t : t->reshape({dim ? t->numel() / dim : 0, dim});
  return Held{dim == 1 || r.stride(1) == 1 ? r : r.contiguous()};
}
struct Norm {
  Held x, residual, weight;
};
template <typename P>
Norm norm_operands(P &p, const at::Tensor &x, const at::Tensor &weight, const at::Tensor *residual, float eps) {
  const int dt = dtype_of(x);
  if (x.dim() < 1 || dt < 0) refuse(PyExc_TypeError, "x must be (..., dim) fp32/fp16/bf16");
  if (x.size(-1) < 1) refuse(PyExc_ValueError, "x must have at least one channel");
  const int wt = dtype_of(weight);
  if (weight.dim() != 1 || weight.size(0) != x.size(-1) || (wt != SS_F32 && wt != dt))
    refuse(PyExc_TypeError, "weight must be (dim,) in x's dtype or float32");
  if (residual && (residual->sizes() != x.sizes() || (dtype_of(*residual) != dt && dtype_of(*residual) != SS_F32)))
    refuse(PyExc_TypeError, "residual must match x in shape, in x's dtype or float32");
  on(&weight, x, "weight");
  on(residual, x, "residual");
  Norm n{rows2(&x), rows2(residual), flat(&weight)};
  p.abi_version = SS_ABI_VERSION;
  p.dtype = dt;
  p.residual_dtype = residual ? dtype_of(*residual) : dt;
  p.weight_dtype = wt;
  p.eps = eps;
  p.dim = x.size(-1);
  p.rows = x.numel() / p.dim;
  p.x = ptr(n.x.get());
  p.residual = ptr(n.residual.get());
  p.weight = ptr(n.weight.get());
  p.x_stride = n.x.t.stride(0);
  p.residual_stride = residual ? n.residual.t.stride(0) : 0;
  p.out_stride = p.sum_stride = p.dim;
  return n;
}

struct Normed {
  at::Tensor out, sum, rstd;
};
Normed norm_forward(const at::Tensor &x, const at::Tensor &weight, const at::Tensor *residual, float eps, bool want_sum, bool want_rstd) {
  ss_rms_norm_params p{};
  const Norm n = norm_operands(p, x, weight, residual, eps);
  const c10::cuda::CUDAGuard guard(x.device());
  Normed r;
  r.out = at::empty(x.sizes(), x.options());
  if (want_sum && residual) r.sum = at::empty(x.sizes(), residual->options());
  if (want_rstd) r.rstd = at::empty({p.rows}, x.options().dtype(at::kFloat));
  p.out = place(r.out);
  p.sum = place(r.sum);
  p.rstd = static_cast<float *>(place(r.rstd));
  check(g_norm(&p, stream_of(x)));
  return r;
}

enum { kNormDx, kNormDweight, kNormDresidual, kNormGrads };
// The gradients that `wanted` has a bit for. Where both have one type, dx and
// dresidual are one tensor.
std::array<at::Tensor, kNormGrads> norm_backward(const at::Tensor &dout, const at::Tensor *dsum, const at::Tensor &sum, const at::Tensor &weight,
                                                 const at::Tensor &rstd, int wanted) {
  ss_rms_norm_bwd_params p{};
  p.dtype = dtype_of(dout);
  p.residual_dtype = dtype_of(sum);
  p.weight_dtype = dtype_of(weight);
  p.dim = dout.size(-1);
  p.rows = dout.numel() / p.dim;
  const Held d = rows2(&dout), ds = rows2(dsum), s = rows2(&sum), w = flat(&weight), rs = flat(&rstd);
  const c10::cuda::CUDAGuard guard(dout.device());
  const bool same = p.residual_dtype == p.dtype, want_x = wanted >> kNormDx & 1, want_res = wanted >> kNormDresidual & 1;
  at::Tensor dx, dres, dw;
  if (want_x || (want_res && same)) dx = at::empty(dout.sizes(), dout.options());
  if (want_res) dres = same ? dx : at::empty(sum.sizes(), sum.options());
  if (wanted >> kNormDweight & 1) dw = at::empty({p.dim}, weight.options());
  p.abi_version = SS_ABI_VERSION;
  p.dout = d.t.data_ptr();
  p.dsum = ptr(ds.get());
  p.sum = ptr(s.get());
  p.weight = ptr(w.get());
  p.rstd = fptr(rs.get());
  p.dx = place(dx);
  p.dresidual = same ? nullptr : place(dres);
  p.dweight = place(dw);
  p.dout_stride = d.t.stride(0);
  p.dsum_stride = ds.get() ? ds.t.stride(0) : 0;
  p.sum_stride = s.t.stride(0);
  p.dx_stride = p.dresidual_stride = p.dim;
  check(g_norm_bwd_ws(&p, &p.workspace_bytes));
  const at::Tensor ws = workspace(p.workspace_bytes, dout);
  p.workspace = place(ws);
  check(g_norm_bwd(&p, stream_of(dout)));
  return {want_x ? dx : at::Tensor(), dw, dres};
}

// rms_norm_fn with its backward, from the kept sum and 1 / rms of each row.
struct RmsNorm : torch::autograd::Function<RmsNorm> {
  static variable_list forward(AutogradContext *ctx, const at::Tensor &x, const at::Tensor &weight, const std::optional<at::Tensor> &residual, double eps) {
    const Normed r = norm_forward(x, weight, some(residual), static_cast<float>(eps), true, true);
    ctx->save_for_backward({r.sum.defined() ? r.sum : x, weight, r.rstd});
    ctx->saved_data["dtype"] = static_cast<int64_t>(x.scalar_type());
    ctx->set_materialize_grads(false);
    return r.sum.defined() ? variable_list{r.out, r.sum} : variable_list{r.out};
  }
  static variable_list backward(AutogradContext *ctx, variable_list d) {
    const variable_list saved = ctx->get_saved_variables();
    variable_list grads(4);
    const bool residual = d.size() > 1;
    if (!d[0].defined() && !(residual && d[1].defined())) return grads;
    int wanted = ctx->needs_input_grad(0) << kNormDx | ctx->needs_input_grad(1) << kNormDweight;
    if (residual) wanted |= ctx->needs_input_grad(2) << kNormDresidual;
    std::array<at::Tensor, kNormGrads> r = on_engine("rms_norm_fn's backward", [&] {
      const at::AutoGradMode off(false);
      const at::Tensor dout =
          d[0].defined() ? d[0] : at::zeros(saved[0].sizes(), saved[0].options().dtype(static_cast<at::ScalarType>(ctx->saved_data["dtype"].toInt())));
      return norm_backward(dout, residual && d[1].defined() ? &d[1] : nullptr, saved[0], saved[1], saved[2], wanted);
    });
    return once("rms_norm_fn", {r[kNormDx], r[kNormDweight], r[kNormDresidual], at::Tensor()});
  }
};

// rms_norm(x, weight, residual, eps, want_sum) -> (out, sum or None)
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 5, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), &weight = need(a[1], "weight"), *residual = opt(a[2], "residual");
    const double eps = number(a[3]);
    const bool want_sum = flag(a[4]);
    no_tangent({&x, &weight, residual});
    if (wants_grad({&x, &weight, residual})) {
      const variable_list r = RmsNorm::apply(x, weight, maybe(residual), eps);
      return tuple_of({r[0], r.size() > 1 ? r[1] : at::Tensor()});
    }
    const Normed r = norm_forward(x, weight, residual, static_cast<float>(eps), want_sum, false);
    return tuple_of({r.out, r.sum});
  });
}

// rms_norm_quant(x, weight, residual, eps, want_sum, group, e8m0) -> (out, scale, sum)
PyObject *rms_norm_quant(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 7, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), &weight = need(a[1], "weight"), *residual = opt(a[2], "residual");
    ss_rms_norm_quant_params p{};
    const Norm n = norm_operands(p, x, weight, residual, static_cast<float>(number(a[3])));
    no_grad({&x, &weight, residual});
    const bool want_sum = flag(a[4]) && residual, e8m0 = flag(a[6]);
    p.group = integer(a[5]);
    if (p.group != 0 && p.group != 32 && p.group != 64 && p.group != 128) refuse(PyExc_ValueError, "group_size must be None, 32, 64 or 128");
    const c10::cuda::CUDAGuard guard(x.device());
    std::vector<int64_t> sizes(x.sizes().begin(), x.sizes().end());
    sizes.back() = p.group ? (p.dim + p.group - 1) / p.group : 1;
    at::Tensor out = at::empty(x.sizes(), x.options().dtype(at::kFloat8_e4m3fn)),
               scale = at::empty(sizes, x.options().dtype(e8m0 ? at::kFloat8_e8m0fnu : at::kFloat)), sum;
    if (want_sum) sum = at::empty(x.sizes(), residual->options());
    p.scale_type = e8m0 ? SS_SCALE_E8M0 : SS_SCALE_F32;
    p.out = out.data_ptr();
    p.scale = scale.data_ptr();
    p.sum = want_sum ? sum.data_ptr() : nullptr;
    check(g_quant(&p, stream_of(x)));
    return tuple_of({out, scale, sum});
  });
}

PyMethodDef g_methods[] = {method<init>("init"),
                           method<gated_scan>("gated_scan"),
                           method<packed_gated_scan>("packed_gated_scan"),
                           method<gated_state_update>("gated_state_update"),
                           method<rms_norm>("rms_norm"),
                           method<rms_norm_quant>("rms_norm_quant"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind(void) { return PyModule_Create(&g_module); }
