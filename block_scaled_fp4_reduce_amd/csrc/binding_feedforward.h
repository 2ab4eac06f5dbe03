// binding_feedforward.h -- the Python calls of the feed-forward operators; part
// of binding.cpp, whose helpers and errors they share.
#pragma once

// x [rows][cols] of this type on the GPU, the values of a row in one run; any
// number of cols with cols < 0.
struct Rows {
  void* p;
  int64_t stride, rows, cols;
};
Rows rows_of(const at::Tensor& x, at::ScalarType type, int64_t rows, int64_t cols, const char* what) {
  if (x.scalar_type() != type)
    fail(PyExc_TypeError, std::string(what) + " must be " + at::toString(type));
  if (!x.is_cuda() || x.dim() != 2 || (rows >= 0 && x.size(0) != rows) ||
      (cols >= 0 && x.size(1) != cols))
    fail(PyExc_ValueError, std::string(what) + " must be a GPU tensor [" +
                               (rows < 0 ? "tokens" : std::to_string(rows)) + "][" +
                               (cols < 0 ? "cols" : std::to_string(cols)) + "], got " + shape_text(x));
  Rows r{x.data_ptr(), x.size(1), x.size(0), x.size(1)};
  if (r.rows && r.cols > 1 && x.stride(1) != 1)
    fail(PyExc_ValueError, std::string(what) + ": the values of a row must be contiguous");
  if (r.rows > 1 && r.cols > 0) r.stride = x.stride(0);
  return r;
}

// An output of the caller's, refused before anything is done.
void given_rows(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols, const char* what) {
  if (o != Py_None) rows_of(tensor(o, what), type, rows, cols, what);
}

const fp4_weights* weights_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) throw PyError{};
  return (const fp4_weights*)p;
}

void* workspace(PyObject* given, size_t need, Stream& st, const at::Tensor& on, at::Tensor& ws) {
  if (given != Py_None) {
    ws = tensor(given, "ws");
    if (!ws.is_cuda() || !ws.is_contiguous())
      fail(PyExc_ValueError, "ws must be a contiguous GPU tensor");
  } else if (need) {
    ws = st.empty({(int64_t)need}, at::kByte, on);
  }
  return ws.defined() ? ws.data_ptr() : nullptr;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> parts) {
  PyObject* r = PyTuple_New((Py_ssize_t)parts.size());
  if (!r) throw PyError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : parts) {
    PyObject* o = Py_None;
    if (t.defined()) o = THPVariable_Wrap(t);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// The weights of a call are on the tensors' device.
void same_device(PyObject* handle, const at::Tensor& x) {
  const int64_t d = device_of(handle);
  if (d >= 0 && x.is_cuda() && x.device().index() != d)
    fail(PyExc_ValueError, "the weights are on another device (cuda:" + std::to_string(d) +
                               ") than the tensors: " + x.device().str());
}

// Neither a tensor nor the alpha of the handle's weights wants a gradient.
void no_backward(const char* name, PyObject* handle, PyObject* const* a, int n) {
  bool wanted = wants_gradient(a, n);
  if (!wanted && !PyLong_CheckExact(handle)) {
    PyObject* alpha = PyObject_GetAttrString(handle, "alpha");
    if (!alpha) throw PyError{};
    wanted = wants_gradient(&alpha, 1);
    Py_DECREF(alpha);
  }
  if (wanted)
    fail(PyExc_RuntimeError, std::string(name) + " has no backward, but a tensor requires a gradient: "
                             "detach it or call under torch.no_grad()");
}

// linear(weights, x, dtype is float32, out, ws, stream) -> out
PyObject* linear(PyObject* const* a) {
  PyObject* const floats[] = {a[1], a[3]};
  no_backward("fp4_linear", a[0], floats, 2);
  const fp4_weights* w = weights_of(a[0]);
  PyObject* const all[] = {a[1], a[3], a[4]};
  one_device(all, 3);
  const at::Tensor& x = tensor(a[1], "x");
  same_device(a[0], x);
  const Rows xr = rows_of(x, at::kBFloat16, -1, w->cols, "x");
  const bool f32 = truth(a[2]);
  const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
  given_rows(a[3], type, xr.rows, w->rows, "out");
  Stream st(a[5], x);
  const at::Tensor out = given_or_new(a[3], "out", st, {xr.rows, w->rows}, type, x);
  const Rows o = rows_of(out, type, xr.rows, w->rows, "out");
  at::Tensor ws;
  void* wp = workspace(a[4], fp4_linear_workspace_bytes(w, xr.rows), st, x, ws);
  check("fp4_linear", fp4_linear(w, (const uint16_t*)xr.p, xr.stride, xr.rows, o.p, o.stride, f32, wp,
                                 ws.defined() ? ws.nbytes() : 0, st.raw()));
  return THPVariable_Wrap(out);
}

// experts(gate_up, down, x, weights, experts, out, ws, stream) -> out
PyObject* experts(PyObject* const* a) {
  PyObject* const floats[] = {a[2], a[3], a[5]};
  no_backward("fp4_experts", a[0], floats, 3);
  no_backward("fp4_experts", a[1], nullptr, 0);
  const fp4_weights *gu = weights_of(a[0]), *dn = weights_of(a[1]);
  PyObject* const all[] = {a[2], a[3], a[4], a[5], a[6]};
  one_device(all, 5);
  const at::Tensor& x = tensor(a[2], "x");
  same_device(a[0], x);
  same_device(a[1], x);
  const Rows xr = rows_of(x, at::kBFloat16, -1, gu->cols, "x");
  const at::Tensor& ids = tensor(a[4], "experts");
  const int64_t k = ids.dim() == 2 ? ids.size(1) : 0;
  const int32_t* ep = array_of<int32_t>(a[4], at::kInt, {xr.rows, k}, "experts");
  const float* wp = array_of<float>(a[3], at::kFloat, {xr.rows, k}, "weights");
  given_rows(a[5], at::kBFloat16, xr.rows, xr.cols, "out");
  Stream st(a[7], x);
  const at::Tensor out = given_or_new(a[5], "out", st, x.sizes(), at::kBFloat16, x);
  const Rows o = rows_of(out, at::kBFloat16, xr.rows, xr.cols, "out");
  at::Tensor ws;
  void* sp = workspace(a[6], fp4_experts_workspace_bytes(gu, dn, xr.rows, k), st, x, ws);
  check("fp4_experts", fp4_experts(gu, dn, (const uint16_t*)xr.p, xr.stride, xr.rows, wp, ep, k,
                                   (uint16_t*)o.p, o.stride, sp, ws.defined() ? ws.nbytes() : 0,
                                   st.raw()));
  return THPVariable_Wrap(out);
}

// experts_ws(gate_up, down, tokens, top_k) -> bytes
PyObject* experts_ws(PyObject* const* a) {
  return PyLong_FromSize_t(
      fp4_experts_workspace_bytes(weights_of(a[0]), weights_of(a[1]), integer(a[2]), integer(a[3])));
}

bool sigmoid_scores(PyObject* o) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (!s) fail(PyExc_TypeError, "scores must be \"softmax\" or \"sigmoid\"");
  if (!strcmp(s, "sigmoid")) return true;
  if (strcmp(s, "softmax")) fail(PyExc_ValueError, "scores must be \"softmax\" or \"sigmoid\"");
  return false;
}

fp4_routing routing_of(PyObject* logits, int64_t top_k, PyObject* scores, PyObject* renormalize,
                       PyObject* scale) {
  const at::Tensor& l = tensor(logits, "logits");
  const bool bf = l.scalar_type() == at::kBFloat16;
  const Rows r = rows_of(l, bf ? at::kBFloat16 : at::kFloat, -1, -1, "logits");
  if (r.cols > INT32_MAX || top_k < 0 || top_k > INT32_MAX)
    fail(PyExc_ValueError, "logits or top_k out of range");
  fp4_routing x = {};
  x.logits = r.p;
  x.stride = r.stride;
  x.tokens = r.rows;
  x.experts = (int32_t)r.cols;
  x.top_k = (int32_t)top_k;
  x.groups = x.top_groups = x.group_top = 1;
  x.sigmoid = sigmoid_scores(scores);
  x.renormalize = truth(renormalize);
  x.logits_bf16 = bf;
  x.scale = (float)number(scale);
  return x;
}

// route(logits, top_k, scores, bias, groups, top_groups, group_top, renormalize, scale, out,
// stream) -> (weights, experts); by way of torch's autograd where logits want a gradient
PyObject* route(PyObject* const* a) {
  PyObject* given[2];
  pair_of(a[9], &given[0], &given[1]);
  if (wants_gradient(a, 1) || wants_gradient(a + 3, 1) || wants_gradient(given, 1)) {
    if (wants_gradient(a + 3, 1))
      fail(PyExc_RuntimeError, "expert_route has no gradient of its bias");
    if (a[9] != Py_None)
      fail(PyExc_RuntimeError, "expert_route: out cannot carry the gradient that logits require");
    PyObject* const args[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[10]};
    return in_package("_expert_route_autograd", args, 10);
  }
  PyObject* const all[] = {a[0], a[3], given[0], given[1]};
  one_device(all, 4);
  fp4_routing x = routing_of(a[0], integer(a[1]), a[2], a[7], a[8]);
  if (a[3] != Py_None) x.bias = array_of<float>(a[3], at::kFloat, {x.experts}, "bias");
  x.groups = integer32(a[4], "groups");
  x.top_groups = integer32(a[5], "top_groups");
  x.group_top = integer32(a[6], "group_top");
  const at::Tensor& l = tensor(a[0], "logits");
  if (given[0] != Py_None) array_of<float>(given[0], at::kFloat, {x.tokens, x.top_k}, "out weights");
  if (given[1] != Py_None) array_of<int32_t>(given[1], at::kInt, {x.tokens, x.top_k}, "out experts");
  Stream st(a[10], l);
  const at::Tensor w = given_or_new(given[0], "weights", st, {x.tokens, x.top_k}, at::kFloat, l);
  const at::Tensor e = given_or_new(given[1], "experts", st, {x.tokens, x.top_k}, at::kInt, l);
  check("expert_route", expert_route(&x, (float*)w.data_ptr(), (int32_t*)e.data_ptr(), st.raw()));
  return pair(w, e);
}

// route_backward(dweights, logits, experts, scores, renormalize, scale, out, stream) -> dlogits
PyObject* route_backward(PyObject* const* a) {
  PyObject* const all[] = {a[0], a[1], a[2], a[6]};
  no_tangent("expert_route_backward", all, 4);
  one_device(all, 4);
  const at::Tensor &l = tensor(a[1], "logits"), &ids = tensor(a[2], "experts");
  const fp4_routing x = routing_of(a[1], ids.dim() == 2 ? ids.size(1) : 0, a[3], a[4], a[5]);
  const int32_t* ep = array_of<int32_t>(a[2], at::kInt, {x.tokens, x.top_k}, "experts");
  const float* gp = array_of<float>(a[0], at::kFloat, {x.tokens, x.top_k}, "dweights");
  given_rows(a[6], l.scalar_type(), x.tokens, x.experts, "out");
  Stream st(a[7], l);
  const at::Tensor d = given_or_new(a[6], "out", st, l.sizes(), l.scalar_type(), l);
  const Rows dr = rows_of(d, l.scalar_type(), x.tokens, x.experts, "out");
  check("expert_route_backward",
        expert_route_backward(&x, gp, ep, dr.p, dr.stride, st.raw()));
  return THPVariable_Wrap(d);
}

// [x, block, weight, block_weight, gate, scale, eps] of a call
fp4_residual residual_of(PyObject* const* a) {
  fp4_residual r = {};
  const Rows x = rows_of(tensor(a[0], "x"), at::kBFloat16, -1, -1, "x");
  const Rows b = rows_of(tensor(a[1], "block"), at::kBFloat16, x.rows, x.cols, "block");
  if (x.cols > INT32_MAX) fail(PyExc_ValueError, "x is out of range");
  r.x = (const uint16_t*)x.p;
  r.block = (const uint16_t*)b.p;
  r.x_stride = x.stride;
  r.block_stride = b.stride;
  r.tokens = x.rows;
  r.dim = (int32_t)x.cols;
  r.weight = array_of<uint16_t>(a[2], at::kBFloat16, {x.cols}, "weight");
  if (a[3] != Py_None)
    r.block_weight = array_of<uint16_t>(a[3], at::kBFloat16, {x.cols}, "block_weight");
  if (a[4] != Py_None) {
    r.token_gate = tensor(a[4], "gate").dim() == 2;
    r.gate = r.token_gate ? array_of<uint16_t>(a[4], at::kBFloat16, {x.rows, 1}, "gate")
                          : array_of<uint16_t>(a[4], at::kBFloat16, {x.cols}, "gate");
  }
  r.scale = (float)number(a[5]);
  r.eps = (float)number(a[6]);
  return r;
}

Rows like_x(const at::Tensor& t, const fp4_residual& r, const char* what) {
  return rows_of(t, at::kBFloat16, r.tokens, r.dim, what);
}

// residual(x, block, weight, block_weight, gate, scale, eps, out, stream) -> (y, z); by way of
// torch's autograd where an input wants a gradient
PyObject* residual(PyObject* const* a) {
  PyObject* given[2];
  pair_of(a[7], &given[0], &given[1]);
  if (wants_gradient(a, 5) || wants_gradient(given, 2)) {
    if (a[7] != Py_None)
      fail(PyExc_RuntimeError, "residual_norm: out cannot carry the gradient that an input requires");
    PyObject* const args[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[8]};
    return in_package("_residual_norm_autograd", args, 8);
  }
  PyObject* const all[] = {a[0], a[1], a[2], a[3], a[4], given[0], given[1]};
  one_device(all, 7);
  const fp4_residual r = residual_of(a);
  const at::Tensor& x = tensor(a[0], "x");
  given_rows(given[0], at::kBFloat16, r.tokens, r.dim, "out y");
  given_rows(given[1], at::kBFloat16, r.tokens, r.dim, "out z");
  Stream st(a[8], x);
  const at::Tensor y = given_or_new(given[0], "out y", st, x.sizes(), at::kBFloat16, x);
  const at::Tensor z = given_or_new(given[1], "out z", st, x.sizes(), at::kBFloat16, x);
  const Rows yr = like_x(y, r, "out y"), zr = like_x(z, r, "out z");
  check("residual_norm", residual_norm(&r, (uint16_t*)yr.p, yr.stride, (uint16_t*)zr.p, zr.stride,
                                       st.raw()));
  return pair(y, z);
}

// residual_backward(dy, dz, x, block, weight, block_weight, gate, scale, eps, out, ws, stream)
// -> (dx, dblock, dblock_weight, dweight, dgate)
PyObject* residual_backward(PyObject* const* a) {
  PyObject* given[2];
  pair_of(a[9], &given[0], &given[1]);
  PyObject* const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], given[0], given[1], a[10]};
  no_tangent("residual_norm_backward", all, 10);
  one_device(all, 10);
  const fp4_residual r = residual_of(a + 2);
  const at::Tensor& x = tensor(a[2], "x");
  const Rows dy = like_x(tensor(a[0], "dy"), r, "dy"), dz = like_x(tensor(a[1], "dz"), r, "dz");
  given_rows(given[0], at::kBFloat16, r.tokens, r.dim, "out dx");
  given_rows(given[1], at::kBFloat16, r.tokens, r.dim, "out dblock");
  Stream st(a[11], x);
  const at::Tensor dx = given_or_new(given[0], "out dx", st, x.sizes(), at::kBFloat16, x);
  const at::Tensor db = given_or_new(given[1], "out dblock", st, x.sizes(), at::kBFloat16, x);
  const Rows dxr = like_x(dx, r, "out dx"), dbr = like_x(db, r, "out dblock");
  at::Tensor dbw, dg, ws;
  const at::Tensor dw = st.empty({r.dim}, at::kFloat, x);
  if (r.block_weight) dbw = st.empty({r.dim}, at::kFloat, x);
  if (r.gate) dg = st.empty(tensor(a[6], "gate").sizes(), at::kFloat, x);
  void* wp = workspace(a[10], residual_norm_workspace_bytes(r.tokens, r.dim), st, x, ws);
  auto floats = [](const at::Tensor& t) { return t.defined() ? (float*)t.data_ptr() : nullptr; };
  check("residual_norm_backward",
        residual_norm_backward(&r, (const uint16_t*)dy.p, dy.stride, (const uint16_t*)dz.p, dz.stride,
                               (uint16_t*)dxr.p, dxr.stride, (uint16_t*)dbr.p, dbr.stride, floats(dbw),
                               floats(dw), floats(dg), wp, ws.defined() ? ws.nbytes() : 0, st.raw()));
  return tuple_of({dx, db, dbw, dw, dg});
}
