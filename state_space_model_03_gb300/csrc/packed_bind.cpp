// Python binding of the packed operators (include/ssfwd_packed.h): argument
// checks, output allocation and the call, in C++ because the one-token
// operators take a few microseconds on the GPU, which marshalling some dozen
// tensors in Python does not keep up with (22 us a call; here a few).
//
// The module does not link against libssfwd.so: init() takes the addresses of
// its entry points, so that whichever build of the library Python has loaded is
// the one that runs.
#include "bind_common.h"

namespace {

int (*g_tables)(const ss_request_tables_params *, void *);
int (*g_conv)(const ss_packed_conv1d_params *, void *);
int (*g_conv_update)(const ss_packed_conv1d_update_params *, void *);
int (*g_scan)(const ss_head_scan_params *, void *);
int (*g_scan_ws)(const ss_head_scan_params *, int64_t *);
int (*g_update)(const ss_head_state_update_params *, void *);

PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    auto at_ = [&](int i) { return reinterpret_cast<void *>(integer(a[i])); };
    g_tables = reinterpret_cast<decltype(g_tables)>(at_(0));
    g_conv = reinterpret_cast<decltype(g_conv)>(at_(1));
    g_conv_update = reinterpret_cast<decltype(g_conv_update)>(at_(2));
    g_scan = reinterpret_cast<decltype(g_scan)>(at_(3));
    g_scan_ws = reinterpret_cast<decltype(g_scan_ws)>(at_(4));
    g_update = reinterpret_cast<decltype(g_update)>(at_(5));
    g_text = reinterpret_cast<decltype(g_text)>(at_(6));
    Py_INCREF(a[7]);
    g_error = a[7];
    Py_RETURN_NONE;
  });
}

// request_tables(lengths, num_tokens, context, slots, free_slots, block) ->
// (offsets, token_request, token_position, blocks, slots, counts, plan, max_blocks, context, carried)
PyObject *request_tables(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 6, [&]() -> PyObject * {
    const at::Tensor &len = need(a[0], "lengths");
    if (len.dim() != 1) refuse(PyExc_TypeError, "lengths must be int32 (requests,)");
    const int64_t n = len.size(0), tokens = integer(a[1]), block = integer(a[5]);
    const Held lengths = int32(&len, "lengths", n, len), context = int32(opt(a[2], "context"), "context", n, len);
    const Held slots = int32(opt(a[3], "slots"), "slots", n, len);
    const at::Tensor *f = opt(a[4], "free_slots");
    if (f && !slots.get()) refuse(PyExc_ValueError, "free_slots goes with slots");
    const Held free = int32(f, "free_slots", f ? f->numel() : 0, len);
    if (tokens < 0 || block < 1) refuse(PyExc_ValueError, "num_tokens must be >= 0 and block >= 1");
    const int64_t most = tokens / block + std::min(n, tokens);
    const c10::cuda::CUDAGuard guard(len.device());
    // one allocation for all tables, each on 16 bytes of it
    const int64_t sizes[7] = {n + 1, tokens, tokens, 4 * most, n, 4, tokens / block};
    int64_t start[8] = {};
    for (int i = 0; i < 7; ++i) start[i + 1] = start[i] + (sizes[i] + 3) / 4 * 4;
    const at::Tensor all = at::empty({start[7]}, len.options());
    int32_t *const base = all.data_ptr<int32_t>();
    auto table = [&](int i) {
      at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
      t.unsafeGetTensorImpl()->set_storage_offset(start[i]);
      if (i == 3) t.unsafeGetTensorImpl()->set_sizes_contiguous({most, 4});
      else t.unsafeGetTensorImpl()->set_sizes_contiguous({sizes[i]});
      return t;
    };
    ss_request_tables_params p{};
    p.abi_version = SS_ABI_VERSION;
    p.requests = n;
    p.tokens = tokens;
    p.block = block;
    p.max_blocks = most;
    p.free = f ? f->numel() : 0;
    p.lengths = iptr(lengths.get());
    p.context = iptr(context.get());
    p.slots = iptr(slots.get());
    p.free_slots = iptr(free.get());
    p.offsets = base + start[0];
    p.token_request = base + start[1];
    p.token_position = base + start[2];
    p.blocks = base + start[3];
    p.carried = base + start[6];
    p.slot_map = base + start[4];
    p.counts = base + start[5];
    check(g_tables(&p, stream_of(len)));
    Plan plan{{n, tokens, block, most, p.offsets, p.token_request, p.blocks, p.carried, p.slot_map, p.counts, p.context}, len.get_device()};
    PyObject *r = PyTuple_New(10);
    if (!r) throw python_error();
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(table(i)));
    PyTuple_SET_ITEM(r, 6, PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&plan), sizeof(plan)));
    PyTuple_SET_ITEM(r, 7, PyLong_FromLongLong(most));
    if (context.get()) {
      PyTuple_SET_ITEM(r, 8, THPVariable_Wrap(context.t));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 8, Py_None);
    }
    PyTuple_SET_ITEM(r, 9, THPVariable_Wrap(table(6)));
    return r;
  });
}

// The operands that both convolutions share; fills everything but rows.
struct Conv {
  Held x, weight, bias;
  int64_t dim, width;
};
template <typename P>
Conv conv_operands(P &p, const at::Tensor &x, const at::Tensor &weight, const at::Tensor *bias, const at::Tensor *state, int64_t act) {
  const int dt = dtype_of(x);
  if (x.dim() != 2 || dt < 0) refuse(PyExc_TypeError, "x must be (tokens, dim) fp32/fp16/bf16");
  const int64_t dim = x.size(1);
  if (weight.dim() != 2 || weight.size(0) != dim || weight.scalar_type() != at::kFloat)
    refuse(PyExc_TypeError, "weight must be float32 (dim, width)");
  const int64_t width = weight.size(1);
  if (bias && (bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != dim))
    refuse(PyExc_TypeError, "bias must be float32 (dim,)");
  if (state) {
    if (state->scalar_type() != x.scalar_type() || state->dim() != 3 || state->size(1) != dim || state->size(2) != width - 1)
      refuse(PyExc_TypeError, "conv_state must be x's dtype (slots, dim, width - 1)");
    if (state->numel() && (state->stride(2) != 1 || state->stride(1) != width - 1))
      refuse(PyExc_ValueError, "conv_state must be contiguous but for its slot stride (it is updated in place)");
  }
  on(&weight, x, "weight");
  on(bias, x, "bias");
  on(state, x, "conv_state");
  no_grad({&x, &weight, bias, state});
  Conv c{rows(&x), flat(&weight), flat(bias), dim, width};
  p.abi_version = SS_ABI_VERSION;
  p.dtype = dt;
  p.activation = static_cast<int32_t>(act);
  p.dim = dim;
  p.width = width;
  p.x = c.x.t.data_ptr();
  p.weight = fptr(c.weight.get());
  p.bias = fptr(c.bias.get());
  p.x_stride = c.x.t.stride(0);
  p.out_stride = dim;
  if (state) {
    p.slots = state->size(0);
    p.conv_state = state->data_ptr();
    p.state_stride = state->stride(0);
  }
  return c;
}

// packed_conv1d(x, weight, plan, bias, conv_state, activation) -> out
PyObject *packed_conv1d(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 6, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x");
    ss_packed_conv1d_params p{};
    const at::Tensor *state = opt(a[4], "conv_state");
    const Conv c = conv_operands(p, x, need(a[1], "weight"), opt(a[3], "bias"), state, integer(a[5]));
    p.tables = plan_of(a[2], x).t;
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options());
    p.out = out.data_ptr();
    check(g_conv(&p, stream_of(x)));
    changed(state);
    return THPVariable_Wrap(std::move(out));
  });
}

// packed_conv1d_update(x, conv_state, weight, bias, slots, activation) -> out
PyObject *packed_conv1d_update(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 6, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), &state = need(a[1], "conv_state");
    ss_packed_conv1d_update_params p{};
    const Conv c = conv_operands(p, x, need(a[2], "weight"), opt(a[3], "bias"), &state, integer(a[5]));
    p.requests = x.size(0);
    const Held slots = int32(opt(a[4], "slots"), "slots", x.size(0), x);
    p.slot_map = iptr(slots.get());
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options());
    p.out = out.data_ptr();
    check(g_conv_update(&p, stream_of(x)));
    changed(&state);
    return THPVariable_Wrap(std::move(out));
  });
}

// The operands that both scans share; fills everything but rows and out.
struct Heads {
  Held x, dt, A, B, C, D, z, bias;
};
template <typename P>
Heads head_operands(P &p, const at::Tensor &x, const at::Tensor &dt, const at::Tensor &A, const at::Tensor &B, const at::Tensor &C,
                    const at::Tensor *D, const at::Tensor *z, const at::Tensor *bias, bool softplus, const at::Tensor *state) {
  const int ty = dtype_of(x);
  if (x.dim() != 3 || ty < 0) refuse(PyExc_TypeError, "x must be (tokens, heads, headdim) fp32/fp16/bf16");
  const int64_t n = x.size(0), heads = x.size(1), headdim = x.size(2);
  if (dt.dim() != 2 || dt.size(0) != n || dt.size(1) != heads || (dt.scalar_type() != x.scalar_type() && dt.scalar_type() != at::kFloat))
    refuse(PyExc_TypeError, "dt must be (tokens, heads) in x's dtype or float32");
  if (B.dim() != 3 || B.size(0) != n || B.scalar_type() != x.scalar_type() || C.sizes() != B.sizes() || C.scalar_type() != x.scalar_type())
    refuse(PyExc_TypeError, "B and C must be (tokens, groups, dstate) in x's dtype");
  if (z && (z->sizes() != x.sizes() || z->scalar_type() != x.scalar_type())) refuse(PyExc_TypeError, "z must match x in shape and dtype");
  const at::Tensor *per_head[3] = {&A, D, bias};
  const char *names[3] = {"A", "D", "dt_bias"};
  for (int i = 0; i < 3; ++i)
    if (per_head[i] && (per_head[i]->scalar_type() != at::kFloat || per_head[i]->dim() != 1 || per_head[i]->size(0) != heads))
      refuse(PyExc_TypeError, std::string(names[i]) + " must be float32 (heads,)");
  const int64_t groups = B.size(1), dstate = B.size(2);
  if (state) {
    const char *form = "state must be float32 (slots, heads, headdim, dstate) with its last two dimensions contiguous";
    if (state->scalar_type() != at::kFloat || state->dim() != 4 || state->size(1) != heads || state->size(2) != headdim ||
        state->size(3) != dstate)
      refuse(PyExc_TypeError, form);
    if (state->numel() && (state->stride(3) != 1 || (headdim > 1 && state->stride(2) != dstate)))
      refuse(PyExc_ValueError, std::string(form) + " (it is updated in place)");
  }
  on(&dt, x, "dt");
  on(&A, x, "A");
  on(&B, x, "B");
  on(&C, x, "C");
  on(D, x, "D");
  on(z, x, "z");
  on(bias, x, "dt_bias");
  on(state, x, "state");
  no_grad({&x, &dt, &A, &B, &C, D, z, bias, state});
  Heads h{rows(&x), Held{dt}, flat(&A), rows(&B), rows(&C), flat(D), rows(z), flat(bias)};
  p.abi_version = SS_ABI_VERSION;
  p.dtype = ty;
  p.dt_dtype = dtype_of(dt);
  p.dt_softplus = softplus;
  p.heads = heads;
  p.headdim = headdim;
  p.dstate = dstate;
  p.ngroups = groups;
  p.x = h.x.t.data_ptr();
  p.dt = dt.data_ptr();
  p.B = h.B.t.data_ptr();
  p.C = h.C.t.data_ptr();
  p.z = ptr(h.z.get());
  p.A = fptr(h.A.get());
  p.D = fptr(h.D.get());
  p.dt_bias = fptr(h.bias.get());
  for (int i = 0; i < 2; ++i) {
    p.x_stride[i] = h.x.t.stride(i);
    p.dt_stride[i] = dt.stride(i);
    p.B_stride[i] = h.B.t.stride(i);
    p.C_stride[i] = h.C.t.stride(i);
    p.z_stride[i] = z ? h.z.t.stride(i) : 0;
  }
  p.out_stride[0] = heads * headdim;
  p.out_stride[1] = headdim;
  if (state) {
    p.slots = state->size(0);
    p.state = static_cast<float *>(state->data_ptr());
    p.state_stride[0] = state->stride(0);
    p.state_stride[1] = state->stride(1);
  }
  return h;
}

// head_scan(x, dt, A, B, C, plan, D, z, dt_bias, dt_softplus, state) -> out
PyObject *head_scan(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 11, [&]() -> PyObject * {
    const at::Tensor &x = need(a[0], "x"), *state = opt(a[10], "state");
    ss_head_scan_params p{};
    const Heads h = head_operands(p, x, need(a[1], "dt"), need(a[2], "A"), need(a[3], "B"), need(a[4], "C"), opt(a[6], "D"),
                                  opt(a[7], "z"), opt(a[8], "dt_bias"), flag(a[9]), state);
    p.tables = plan_of(a[5], x).t;
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options()), ws;
    p.out = out.data_ptr();
    check(g_scan_ws(&p, &p.workspace_bytes));
    if (p.workspace_bytes > 0) {
      ws = at::empty({p.workspace_bytes}, x.options().dtype(at::kByte));
      p.workspace = ws.data_ptr();
    }
    check(g_scan(&p, stream_of(x)));
    changed(state);
    return THPVariable_Wrap(std::move(out));
  });
}

// head_state_update(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, slots) -> out
PyObject *head_state_update(PyObject *, PyObject *const *a, Py_ssize_t given) {
  return guarded(given, 11, [&]() -> PyObject * {
    const at::Tensor &x = need(a[1], "x"), &state = need(a[0], "state");
    ss_head_state_update_params p{};
    const Heads h = head_operands(p, x, need(a[2], "dt"), need(a[3], "A"), need(a[4], "B"), need(a[5], "C"), opt(a[6], "D"),
                                  opt(a[7], "z"), opt(a[8], "dt_bias"), flag(a[9]), &state);
    p.requests = x.size(0);
    const Held slots = int32(opt(a[10], "slots"), "slots", x.size(0), x);
    p.slot_map = iptr(slots.get());
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out = at::empty(x.sizes(), x.options());
    p.out = out.data_ptr();
    check(g_update(&p, stream_of(x)));
    changed(&state);
    return THPVariable_Wrap(std::move(out));
  });
}

PyMethodDef g_methods[] = {method<init>("init"),
                           method<request_tables>("request_tables"),
                           method<packed_conv1d>("packed_conv1d"),
                           method<packed_conv1d_update>("packed_conv1d_update"),
                           method<head_scan>("head_scan"),
                           method<head_state_update>("head_state_update"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_packed_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__packed_bind(void) { return PyModule_Create(&g_module); }
