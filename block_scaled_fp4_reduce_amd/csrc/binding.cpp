// binding.cpp -- the Python calls of the FP4 cache, its attention, the norm with
// rotation and the feed-forward operators (binding_feedforward.h): checks of the
// tensors, allocation of outputs and workspace, and the call into libfp4q.so.
// These calls are short (a decoding step's kernels take microseconds), so their
// checks run here rather than in Python: the norm of one decoding batch takes 5.5 us a call (17.3 through ctypes and torch.empty).
//
// Errors: TypeError for a wrong dtype, ValueError for a wrong shape, layout or
// device, Fp4Error for a status of the library, RuntimeError where a gradient
// would be lost.
#include <Python.h>

#include <cstring>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp4q.h"

namespace {

struct PyError {};                       // a Python error is set

[[noreturn]] void fail(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw PyError{};
}

std::string shape_text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); i++) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError{};
  return v != 0;
}
int32_t integer32(PyObject* o, const char* what) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) fail(PyExc_ValueError, std::string(what) + " is out of range");
  return (int32_t)v;
}

// x [tokens][heads][dim] bf16 on the GPU, each token's heads in one run.
struct Heads {
  uint16_t* p;
  int64_t stride, tokens, heads, dim;
};
Heads heads_of(const at::Tensor& x, int64_t heads, int64_t dim, const char* what) {
  if (x.scalar_type() != at::kBFloat16)
    fail(PyExc_TypeError, std::string(what) + " must be bfloat16");
  if (!x.is_cuda() || x.dim() != 3 || (heads >= 0 && x.size(1) != heads) ||
      (dim >= 0 && x.size(2) != dim))
    fail(PyExc_ValueError, std::string(what) + " must be a GPU tensor [tokens][heads][dim], got " +
                               shape_text(x));
  Heads h{(uint16_t*)x.data_ptr(), x.size(1) * x.size(2), x.size(0), x.size(1), x.size(2)};
  if (h.tokens && ((h.heads > 1 && x.stride(1) != h.dim) || (h.dim > 1 && x.stride(2) != 1)))
    fail(PyExc_ValueError, std::string(what) + ": a token's heads must be contiguous");
  if (h.tokens > 1) h.stride = x.stride(0);
  return h;
}
Heads heads_of(PyObject* o, int64_t heads, int64_t dim, const char* what) {
  return heads_of(tensor(o, what), heads, dim, what);
}

// A contiguous GPU tensor of this type and shape.
template <typename T>
T* array_of(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  const at::Tensor& x = tensor(o, what);
  if (x.scalar_type() != type)
    fail(PyExc_TypeError, std::string(what) + " must be " + at::toString(type));
  if (!x.is_cuda() || !x.is_contiguous() || x.sizes() != shape) {
    std::string s;
    for (int64_t n : shape) s += "[" + std::to_string(n) + "]";
    fail(PyExc_ValueError, std::string(what) + " must be a contiguous GPU tensor " + s + ", got " +
                               shape_text(x));
  }
  return (T*)x.data_ptr();
}

// The stream of a call: None takes the current one of the tensors' device.
struct Stream {
  c10::DeviceGuard guard;
  c10::hip::HIPStream stream;
  bool given;
  static c10::hip::HIPStream of(PyObject* o, c10::Device dev) {
    if (o == Py_None) return c10::hip::getCurrentHIPStream(dev.index());
    PyObject* raw = PyObject_HasAttrString(o, "cuda_stream")
                        ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!raw) throw PyError{};
    void* p = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw PyError{};
    return c10::hip::getStreamFromExternal((hipStream_t)p, dev.index());
  }
  Stream(PyObject* o, const at::Tensor& on)
      : guard(on.device()), stream(of(o, on.device())), given(o != Py_None) {}
  // New tensors come from the memory of the stream that writes them: what
  // another stream freed may still be in use there.  The caller's current
  // stream, which reads them later, holds them back from reuse.
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& on) {
    const at::TensorOptions options = on.options().dtype(type);
    const c10::hip::HIPStream current = c10::hip::getCurrentHIPStream(stream.device_index());
    if (!given || stream == current) return at::empty(shape, options);
    const c10::hip::HIPStreamGuard there(stream);
    at::Tensor t = at::empty(shape, options);
    if (t.numel()) c10::hip::HIPCachingAllocator::recordStream(t.storage().data_ptr(), current);
    return t;
  }
  void* raw() { return (void*)stream.stream(); }
};

void check(const char* fn, int status) {
  if (status == FP4_OK) return;
  PyObject* m = PyImport_ImportModule("block_scaled_fp4_reduce_amd");
  PyObject* cls = m ? PyObject_GetAttrString(m, "Fp4Error") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "si", fn, status) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(m);
  throw PyError{};
}

// Whether one of the tensors among a[0 .. n - 1] has a tangent of forward-mode
// differentiation (which torch.no_grad leaves on).  Most tensors have no state of
// autograd at all, which is seen without a call (0.1 us of a norm's 5).
bool has_tangent(PyObject* const* a, int n) {
  for (int i = 0; i < n; i++) {
    if (!THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.unsafeGetTensorImpl()->autograd_meta() && t._fw_grad(0).defined())
      return c10::AutogradState::get_tls_state().get_fw_grad_mode();
  }
  return false;
}

// Whether one of them requires a gradient, in grad mode, or has a tangent.
bool wants_gradient(PyObject* const* a, int n) {
  if (at::GradMode::is_enabled())
    for (int i = 0; i < n; i++)
      if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad()) return true;
  return has_tangent(a, n);
}

// The calls of gradients have no derivative of their own.
void no_tangent(const char* name, PyObject* const* a, int n) {
  if (has_tangent(a, n))
    fail(PyExc_RuntimeError, std::string(name) + " has no derivative, but a tensor carries a "
                             "forward-mode gradient");
}

// The caller's tensor, which counts as modified from here on, or a new one.
at::Tensor given_or_new(PyObject* o, const char* what, Stream& st, at::IntArrayRef shape,
                        at::ScalarType type, const at::Tensor& on) {
  if (o == Py_None) return st.empty(shape, type, on);
  const at::Tensor& t = tensor(o, what);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return t;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) throw PyError{};
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// The elements of a pair given by the caller, or None twice.
void pair_of(PyObject* o, PyObject** a, PyObject** b) {
  *a = *b = Py_None;
  if (o == Py_None) return;
  if (!PyTuple_Check(o) && !PyList_Check(o)) fail(PyExc_TypeError, "out must be a pair of tensors");
  if (PySequence_Size(o) != 2) fail(PyExc_ValueError, "out must be a pair of tensors");
  *a = PySequence_Fast_GET_ITEM(o, 0);   // borrowed: a list or tuple
  *b = PySequence_Fast_GET_ITEM(o, 1);
}

// The kernels of a call run on one device, on memory of that device: its tensors
// among a[0 .. n - 1], and those of the cache (an index, -1: not known).
void one_device(PyObject* const* a, int n, int64_t cache = -1) {
  const at::Tensor* first = nullptr;
  for (int i = 0; i < n; i++) {
    if (!THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!first) first = &t;
    if (t.device() != first->device())
      fail(PyExc_ValueError, "tensors of one call on different devices: " + first->device().str() +
                                 " and " + t.device().str());
  }
  if (first && cache >= 0 && first->is_cuda() && first->device().index() != cache)
    fail(PyExc_ValueError, "the cache is on another device (cuda:" + std::to_string(cache) +
                               ") than the tensors: " + first->device().str());
}

// The handle's own struct, from its address; and the device that an address
// knows.
const fp4_kv_cache* cache_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) throw PyError{};
  return (const fp4_kv_cache*)p;
}
int64_t device_of(PyObject* o) {
  if (PyLong_CheckExact(o)) return -1;
  PyObject* d = PyObject_GetAttrString(o, "device_index");
  if (!d) throw PyError{};
  const int64_t i = PyLong_AsLongLong(d);
  Py_DECREF(d);
  if (i == -1 && PyErr_Occurred()) throw PyError{};
  return i;
}

// kv_write(cache, k, v, slots, stream)
PyObject* kv_write(PyObject* const* a) {
  const fp4_kv_cache* c = cache_of(a[0]);
  one_device(a + 1, 3, device_of(a[0]));
  const Heads k = heads_of(a[1], c->heads, c->head_dim, "k"), v = heads_of(a[2], c->heads, c->head_dim, "v");
  if (v.tokens != k.tokens) fail(PyExc_ValueError, "k and v disagree on the number of tokens");
  const int64_t* slots = array_of<int64_t>(a[3], at::kLong, {k.tokens}, "slots");
  Stream st(a[4], tensor(a[1], "k"));
  check("fp4_kv_write", fp4_kv_write(c, k.p, k.stride, v.p, v.stride, slots, k.tokens, st.raw()));
  Py_RETURN_NONE;
}

// kv_read(cache, slots, out, stream) -> (k, v)
PyObject* kv_read(PyObject* const* a) {
  const fp4_kv_cache* c = cache_of(a[0]);
  const at::Tensor& s = tensor(a[1], "slots");
  const int64_t n = s.dim() ? s.size(0) : 0;
  PyObject* all[] = {a[1], nullptr, nullptr};
  pair_of(a[2], &all[1], &all[2]);
  one_device(all, 3, device_of(a[0]));
  const int64_t* slots = array_of<int64_t>(a[1], at::kLong, {n}, "slots");
  Stream st(a[3], s);
  const at::Tensor k = given_or_new(all[1], "k", st, {n, c->heads, c->head_dim}, at::kBFloat16, s);
  const at::Tensor v = given_or_new(all[2], "v", st, {n, c->heads, c->head_dim}, at::kBFloat16, s);
  const Heads hk = heads_of(k, c->heads, c->head_dim, "k"), hv = heads_of(v, c->heads, c->head_dim, "v");
  if (hk.tokens != n || hv.tokens != n)
    fail(PyExc_ValueError, "k, v and slots disagree on the number of tokens");
  check("fp4_kv_read", fp4_kv_read(c, slots, n, hk.p, hk.stride, hv.p, hv.stride, st.raw()));
  return pair(k, v);
}

// [q, page_table, kv_lens, cu_q, max_q, scale, softcap, window] of a call
fp4_kv_queries queries_of(const fp4_kv_cache* c, PyObject* const* a) {
  fp4_kv_queries x;
  const Heads q = heads_of(a[0], -1, c->head_dim, "q");
  const at::Tensor &pt = tensor(a[1], "page_table"), &lens = tensor(a[2], "kv_lens");
  const int64_t seqs = lens.dim() ? lens.size(0) : 0;
  x.kv_lens = array_of<int32_t>(a[2], at::kInt, {seqs}, "kv_lens");
  if (pt.dim() != 2) fail(PyExc_ValueError, "page_table must be [seqs][pages of the longest]");
  x.page_table = array_of<int32_t>(a[1], at::kInt, {seqs, pt.size(1)}, "page_table");
  x.cu_q = a[3] == Py_None ? nullptr : array_of<int32_t>(a[3], at::kInt, {seqs + 1}, "cu_q");
  x.q = q.p;
  x.q_stride = q.stride;
  x.tokens = q.tokens;
  x.seqs = seqs;
  x.max_q = integer(a[4]);
  x.table_width = pt.size(1);
  x.q_heads = (int32_t)q.heads;
  x.window = integer32(a[7], "window");
  x.scale = a[5] == Py_None ? 1.0f / std::sqrt((float)c->head_dim) : (float)number(a[5]);
  x.softcap = (float)number(a[6]);
  return x;
}

// kv_attention_ws(cache, [queries]) -> bytes
PyObject* kv_attention_ws(PyObject* const* a) {
  const fp4_kv_cache* c = cache_of(a[0]);
  one_device(a + 1, 4, device_of(a[0]));
  const fp4_kv_queries x = queries_of(c, a + 1);
  c10::DeviceGuard guard(tensor(a[1], "q").device());
  return PyLong_FromSize_t(fp4_kv_attention_workspace_bytes(c, &x));
}

// kv_attention(cache, [queries], want_lse, out, lse, ws, stream) -> out or (out, lse)
PyObject* kv_attention(PyObject* const* a) {
  PyObject* const floats[] = {a[1], a[10], a[11]};
  if (wants_gradient(floats, 3))
    fail(PyExc_RuntimeError, "fp4_kv_attention has no backward, but a tensor requires a gradient: "
                             "detach it or call under torch.no_grad()");
  const fp4_kv_cache* c = cache_of(a[0]);
  PyObject* const all[] = {a[1], a[2], a[3], a[4], a[10], a[11], a[12]};
  one_device(all, 7, device_of(a[0]));
  const fp4_kv_queries x = queries_of(c, a + 1);
  const at::Tensor& q = tensor(a[1], "q");
  Stream st(a[13], q);
  const at::Tensor out = given_or_new(a[10], "out", st, q.sizes(), at::kBFloat16, q);
  const Heads o = heads_of(out, x.q_heads, c->head_dim, "out");
  if (o.tokens != x.tokens) fail(PyExc_ValueError, "out and q disagree on the number of tokens");
  at::Tensor lse;
  if (a[11] != Py_None) {
    array_of<float>(a[11], at::kFloat, {x.tokens, x.q_heads}, "lse");
    lse = given_or_new(a[11], "lse", st, {}, at::kFloat, q);
  } else if (truth(a[9])) {
    lse = st.empty({x.tokens, x.q_heads}, at::kFloat, q);
  }
  at::Tensor ws;
  if (a[12] != Py_None) {
    ws = tensor(a[12], "ws");
    if (!ws.is_cuda() || !ws.is_contiguous())
      fail(PyExc_ValueError, "ws must be a contiguous GPU tensor");
  } else if (const size_t need = fp4_kv_attention_workspace_bytes(c, &x)) {
    ws = st.empty({(int64_t)need}, at::kByte, q);
  }
  check("fp4_kv_attention",
        fp4_kv_attention(c, &x, o.p, o.stride, lse.defined() ? (float*)lse.data_ptr() : nullptr,
                         ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                         st.raw()));
  return lse.defined() ? pair(out, lse) : THPVariable_Wrap(out);
}

// [q, k, q_weight, k_weight, positions, table, eps, interleaved] of a call
fp4_qk_rope rope_of(PyObject* const* a) {
  fp4_qk_rope x;
  const Heads q = heads_of(a[0], -1, -1, "q"), k = heads_of(a[1], -1, q.dim, "k");
  if (k.tokens != q.tokens) fail(PyExc_ValueError, "q and k disagree on the number of tokens");
  if (q.heads > INT32_MAX || k.heads > INT32_MAX || q.dim > INT32_MAX)
    fail(PyExc_ValueError, "q and k are out of range");
  auto weight = [&](PyObject* o, const char* what) -> const uint16_t* {
    return o == Py_None ? nullptr : array_of<uint16_t>(o, at::kBFloat16, {q.dim}, what);
  };
  x.q_weight = weight(a[2], "q_weight");
  x.k_weight = weight(a[3], "k_weight");
  x.positions = array_of<int64_t>(a[4], at::kLong, {q.tokens}, "positions");
  const at::Tensor& t = tensor(a[5], "table");
  if (t.dim() != 3) fail(PyExc_ValueError, "table must be [positions][rot_dim/2][2]");
  if (t.size(1) > q.dim) fail(PyExc_ValueError, "table has more pairs than a head");
  x.table = array_of<float>(a[5], at::kFloat, {t.size(0), t.size(1), 2}, "table");
  x.q = q.p;
  x.k = k.p;
  x.q_stride = q.stride;
  x.k_stride = k.stride;
  x.tokens = q.tokens;
  x.table_rows = t.size(0);
  x.q_heads = (int32_t)q.heads;
  x.k_heads = (int32_t)k.heads;
  x.head_dim = (int32_t)q.dim;
  x.rot_dim = (int32_t)(2 * t.size(1));
  x.eps = (float)number(a[6]);
  x.flags = truth(a[7]) ? FP4_ROPE_INTERLEAVED : 0;
  return x;
}

Heads like(const at::Tensor& t, const fp4_qk_rope& x, int64_t heads, const char* what) {
  const Heads h = heads_of(t, heads, x.head_dim, what);
  if (h.tokens != x.tokens) fail(PyExc_ValueError, std::string(what) + " has another number of tokens");
  return h;
}

// A function of the package, called with n positional arguments.
PyObject* in_package(const char* name, PyObject* const* a, int n) {
  PyObject* m = PyImport_ImportModule("block_scaled_fp4_reduce_amd");
  PyObject* f = m ? PyObject_GetAttrString(m, name) : nullptr;
  PyObject* r = f ? PyObject_Vectorcall(f, a, n, nullptr) : nullptr;
  Py_XDECREF(f);
  Py_XDECREF(m);
  if (!r) throw PyError{};
  return r;
}

// norm_rope([rope], out, stream) -> (q, k); by way of torch's autograd where
// an input wants a gradient
PyObject* norm_rope(PyObject* const* a) {
  PyObject* given[2];
  pair_of(a[8], &given[0], &given[1]);
  if (wants_gradient(a, 6) || wants_gradient(given, 2)) {
    if (wants_gradient(a + 5, 1))
      fail(PyExc_RuntimeError, "qk_norm_rope has no gradient of its table");
    if (a[8] != Py_None)
      fail(PyExc_RuntimeError, "qk_norm_rope: out cannot carry the gradient that an input requires");
    PyObject* const args[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[9]};
    return in_package("_norm_rope_autograd", args, 9);
  }
  PyObject* const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], given[0], given[1]};
  one_device(all, 8);
  const fp4_qk_rope x = rope_of(a);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  Stream st(a[9], q);
  const at::Tensor yq = given_or_new(given[0], "out q", st, q.sizes(), at::kBFloat16, q);
  const at::Tensor yk = given_or_new(given[1], "out k", st, k.sizes(), at::kBFloat16, k);
  const Heads hq = like(yq, x, x.q_heads, "out q"), hk = like(yk, x, x.k_heads, "out k");
  check("qk_norm_rope", qk_norm_rope(&x, hq.p, hq.stride, hk.p, hk.stride, st.raw()));
  return pair(yq, yk);
}

// norm_rope_backward(dq_out, dk_out, [rope], out, ws, stream) -> (dq, dk, dq_weight, dk_weight)
PyObject* norm_rope_backward(PyObject* const* a) {
  PyObject* given[2];
  pair_of(a[10], &given[0], &given[1]);
  PyObject* const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[11], given[0], given[1]};
  no_tangent("qk_norm_rope_backward", all, 11);
  one_device(all, 11);
  const fp4_qk_rope x = rope_of(a + 2);
  const at::Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k");
  const Heads gq = like(tensor(a[0], "dq_out"), x, x.q_heads, "dq_out");
  const Heads gk = like(tensor(a[1], "dk_out"), x, x.k_heads, "dk_out");
  Stream st(a[12], q);
  const at::Tensor dq = given_or_new(given[0], "out dq", st, q.sizes(), at::kBFloat16, q);
  const at::Tensor dk = given_or_new(given[1], "out dk", st, k.sizes(), at::kBFloat16, k);
  const Heads hq = like(dq, x, x.q_heads, "out dq"), hk = like(dk, x, x.k_heads, "out dk");
  at::Tensor dqw, dkw, ws;
  if (x.q_weight) dqw = st.empty({x.head_dim}, at::kFloat, q);
  if (x.k_weight) dkw = st.empty({x.head_dim}, at::kFloat, q);
  if (a[11] != Py_None) {
    ws = tensor(a[11], "ws");
    if (!ws.is_cuda() || !ws.is_contiguous())
      fail(PyExc_ValueError, "ws must be a contiguous GPU tensor");
  } else if (dqw.defined() || dkw.defined()) {
    ws = st.empty({(int64_t)qk_norm_rope_workspace_bytes(x.head_dim)}, at::kByte, q);
  }
  auto floats = [](const at::Tensor& t) { return t.defined() ? (float*)t.data_ptr() : nullptr; };
  check("qk_norm_rope_backward",
        qk_norm_rope_backward(&x, gq.p, gq.stride, gk.p, gk.stride, hq.p, hq.stride, hk.p, hk.stride,
                              floats(dqw), floats(dkw), ws.defined() ? ws.data_ptr() : nullptr,
                              ws.defined() ? ws.nbytes() : 0, st.raw()));
  PyObject* r = PyTuple_New(4);
  if (!r) throw PyError{};
  const at::Tensor* parts[] = {&dq, &dk, &dqw, &dkw};
  for (int i = 0; i < 4; i++) {
    PyObject* o = Py_None;
    if (parts[i]->defined()) o = THPVariable_Wrap(*parts[i]);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

#include "binding_feedforward.h"

// Calls take exactly N positional arguments; C++ exceptions end here.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define FP4Q_ENTRY(name, n) \
  {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FP4Q_ENTRY(kv_write, 5),      FP4Q_ENTRY(kv_read, 4),   FP4Q_ENTRY(kv_attention_ws, 9),
    FP4Q_ENTRY(kv_attention, 14), FP4Q_ENTRY(norm_rope, 10), FP4Q_ENTRY(norm_rope_backward, 13),
    FP4Q_ENTRY(linear, 6),        FP4Q_ENTRY(experts, 8),   FP4Q_ENTRY(experts_ws, 4),
    FP4Q_ENTRY(route, 11),        FP4Q_ENTRY(route_backward, 8), FP4Q_ENTRY(residual, 9),
    FP4Q_ENTRY(residual_backward, 12),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
