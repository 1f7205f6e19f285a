// The host side of the layer's calls from Python: argument checks and the call of
// the C entry, on tensors as they are.  Through ctypes a call of eleven tensors
// spends 12 us in checks and conversions, several times its kernel; here 0.6 to 0.9, of
// the 3.0 to 3.6 that a call takes with its launch.
// The order of the arguments stands at each entry.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "mla_layer_ops.h"

namespace {

// The C entries, of the library that is loaded already.
decltype(&mla_head_product) head_product_entry;
decltype(&mla_prefill_run) prefill_run_entry;
decltype(&mla_norm_rope_write) norm_rope_write_entry;

struct Refused {};  // the Python error is set

[[noreturn]] void refuse(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused();
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(PyExc_TypeError, std::string(name) + " is needed");
  return *t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
// An integer that the C entry takes as int: what does not fit becomes one that it refuses.
int narrow(PyObject* o) {
  const int64_t v = integer(o);
  return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : int(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return float(v);
}
void* stream_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

int dtype_code(const at::Tensor& t, const char* name, bool with_fp32) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MTV_DTYPE_BF16;
    case at::kHalf: return MTV_DTYPE_FP16;
    case at::kFloat:
      if (with_fp32) return MTV_DTYPE_FP32;
      break;
    default: break;
  }
  refuse(PyExc_TypeError, std::string(name) + " must be bfloat16 or float16" + (with_fp32 ? " or float32" : "") + ", got " +
                              c10::toString(t.scalar_type()));
}
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  return int(t.get_device());
}
void check_kind(const at::Tensor& t, at::ScalarType type, int device, const char* name) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (device_of(t, name) != device) refuse(PyExc_ValueError, std::string(name) + " is on another device");
}
void check_shape(const at::Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

// A contiguous tensor of `count` elements (-1: any).
void* dense(const at::Tensor* t, at::ScalarType type, int device, const char* name, int64_t count = -1) {
  if (!t) return nullptr;
  check_kind(*t, type, device, name);
  if (!t->is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  if (count >= 0 && t->numel() != count)
    refuse(PyExc_ValueError, std::string(name) + " must hold " + std::to_string(count) + " elements, got " +
                                 std::to_string(t->numel()));
  return t->data_ptr();
}

struct View {
  void* at = nullptr;
  int64_t tok = 0, head = 0;
};
// What an empty tensor gives for its address: one that no kernel reads, but not NULL, by which the C entries know an
// argument that is left out.
void* const kNothing = reinterpret_cast<void*>(256);
// A [tokens, heads, dim] or [tokens, dim] view, dense in its last dimension.
View view(const at::Tensor& t, at::ScalarType type, int device, const char* name, at::IntArrayRef shape) {
  check_kind(t, type, device, name);
  check_shape(t, shape, name);
  if (t.stride(-1) != 1 && shape.back() > 1)
    refuse(PyExc_ValueError, std::string(name) + " must be dense in its last dimension");
  return {t.numel() ? t.data_ptr() : kNothing, t.stride(0), shape.size() == 3 ? t.stride(1) : 0};
}

// Other Python threads run during the C call: it may wait for a full queue, and the
// stream for a host function that such a thread has to finish.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F> PyObject* guarded(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(body(a));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// x, w, out, err, stream
PyObject* head_product(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 5, [](PyObject* const* a) -> int {
    const at::Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w"), &out = needed(a[2], "out");
    const int code = dtype_code(x, "x", false);
    const at::ScalarType type = x.scalar_type();
    if (x.dim() != 3 || w.dim() != 3) refuse(PyExc_ValueError, "x must be [tokens, heads, k] and w [heads, k, n]");
    const int64_t tokens = x.size(0), heads = x.size(1), k = x.size(2), cols = w.size(2);
    const int device = device_of(x, "x");
    const View vx = view(x, type, device, "x", {tokens, heads, k}), vo = view(out, type, device, "out", {tokens, heads, cols});
    check_kind(w, type, device, "w");
    check_shape(w, {heads, k, cols}, "w");
    uint32_t* err = static_cast<uint32_t*>(dense(tensor(a[3], "err"), at::kInt, device, "err"));
    void* stream = stream_of(a[4]);
    if (heads > INT32_MAX || k > INT32_MAX || cols > INT32_MAX) return MTV_E_BAD_ARGUMENT;
    const Unlocked unlocked;
    return head_product_entry(vx.at, vx.tok, vx.head, w.data_ptr(), w.stride(0), w.stride(1), w.stride(2), vo.at, vo.tok, vo.head,
                            tokens, int(heads), int(k), int(cols), code, err, stream);
  });
}

// q, k_nope, k_rope, v, qo_indptr, kv_indptr, max_q, max_kv, scale, out, lse, causal, nsplit, workspace, err, stream
PyObject* prefill_run(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 16, [](PyObject* const* a) -> int {
    const at::Tensor &q = needed(a[0], "q"), &kn = needed(a[1], "k_nope"), &kr = needed(a[2], "k_rope"), &v = needed(a[3], "v");
    const at::Tensor &qo = needed(a[4], "qo_indptr"), &kv = needed(a[5], "kv_indptr"), &out = needed(a[9], "out");
    const int code = dtype_code(q, "q", false);
    const at::ScalarType type = q.scalar_type();
    if (q.dim() != 3 || kn.dim() != 3)
      refuse(PyExc_ValueError, "q must be [rows, heads, 192] and k_nope [keys, heads, 128]");
    const int device = device_of(q, "q");
    const int64_t rows = q.size(0), heads = q.size(1), keys = kn.size(0), bs = qo.numel() - 1;
    if (bs < 0) refuse(PyExc_ValueError, "qo_indptr must hold one element more than there are requests");
    const View vq = view(q, type, device, "q", {rows, heads, 192}), vk = view(kn, type, device, "k_nope", {keys, heads, 128});
    const View vv = view(v, type, device, "v", {keys, heads, 128}), vr = view(kr, type, device, "k_rope", {keys, 64});
    const View vo = view(out, type, device, "out", {rows, heads, 128});
    const auto* qp = static_cast<const int64_t*>(dense(&qo, at::kLong, device, "qo_indptr"));
    const auto* kp = static_cast<const int32_t*>(dense(&kv, at::kInt, device, "kv_indptr", bs + 1));
    float* lse = static_cast<float*>(dense(tensor(a[10], "lse"), at::kFloat, device, "lse", rows * heads));
    const at::Tensor* ws = tensor(a[13], "workspace");
    void* wp = dense(ws, at::kByte, device, "workspace");
    uint32_t* err = static_cast<uint32_t*>(dense(tensor(a[14], "err"), at::kInt, device, "err"));
    const int64_t max_q = integer(a[6]), max_kv = integer(a[7]);
    const float scale = real(a[8]);
    const int causal = PyObject_IsTrue(a[11]), nsplit = narrow(a[12]);
    if (causal < 0) throw Refused();
    void* stream = stream_of(a[15]);
    if (bs > INT32_MAX || heads > INT32_MAX) return MTV_E_BAD_ARGUMENT;
    const Unlocked unlocked;
    return prefill_run_entry(vq.at, vq.tok, vq.head, vk.at, vk.tok, vk.head, vr.at, vr.tok, vv.at, vv.tok, vv.head, qp, kp, int(bs),
                           max_q, max_kv, rows, keys, int(heads), code, scale, causal, vo.at, vo.tok, vo.head, lse, nsplit, wp,
                           ws ? uint64_t(ws->numel()) : 0, err, stream);
  });
}

// turns, positions, eps, layout, amplitude, q_in, q_weight, q_nope, q_rope, c_in, c_weight, k_in, out_cache_loc, kv_pool,
// num_valid, err, stream
PyObject* norm_rope_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 17, [](PyObject* const* a) -> int {
    const at::Tensor &turns = needed(a[0], "turns"), &positions = needed(a[1], "positions");
    const at::Tensor *q = tensor(a[5], "q_in"), *qw = tensor(a[6], "q_weight"), *qn = tensor(a[7], "q_nope"), *qr = tensor(a[8], "q_rope");
    const at::Tensor *c = tensor(a[9], "c_in"), *cw = tensor(a[10], "c_weight"), *k = tensor(a[11], "k_in");
    const at::Tensor *loc = tensor(a[12], "out_cache_loc"), *pool = tensor(a[13], "kv_pool"), *valid = tensor(a[14], "num_valid");
    if (!q != !qr) refuse(PyExc_ValueError, "q_in and q_rope go together");
    const at::Tensor* some = q ? q : c;
    if (!some) refuse(PyExc_ValueError, "neither q_in nor c_in is given");
    const char* name = q ? "q_in" : "c_in";
    const int code = dtype_code(*some, name, true);
    const at::ScalarType type = some->scalar_type();
    if (valid && valid->numel() != 1) refuse(PyExc_ValueError, "num_valid must hold one element");
    const int device = device_of(*some, name);
    const int64_t tokens = positions.numel(), rope_dim = 2 * turns.numel();
    View vq, vn, vr, vc, vk;
    int64_t heads = 0, nope = 0, slots = 0;
    if (q) {
      if (q->dim() != 3 || q->size(2) < rope_dim) refuse(PyExc_ValueError, "q_in must be [tokens, heads, nope + rope_dim]");
      heads = q->size(1), nope = q->size(2) - rope_dim;
      vq = view(*q, type, device, "q_in", {tokens, heads, nope + rope_dim});
      vr = view(*qr, type, device, "q_rope", {tokens, heads, rope_dim});
      if ((qn != nullptr) != (qw && nope > 0)) refuse(PyExc_ValueError, "q_nope goes with q_weight");
      if (qn) vn = view(*qn, type, device, "q_nope", {tokens, heads, nope});
    } else if (qn || qw) {
      refuse(PyExc_ValueError, "q_weight and q_nope need q_in");
    }
    const int64_t* lp = nullptr;
    void* pp = nullptr;
    if (pool || c || k || loc || cw) {
      if (!pool || !c || !k || !loc) refuse(PyExc_ValueError, "kv_pool, c_in, k_in and out_cache_loc go together");
      slots = pool->dim() > 0 ? pool->size(0) : 0;
      if (slots == 0) refuse(PyExc_ValueError, "kv_pool is empty");
      vc = view(*c, type, device, "c_in", {tokens, 512});
      vk = view(*k, type, device, "k_in", {tokens, 64});
      lp = static_cast<const int64_t*>(dense(loc, at::kLong, device, "out_cache_loc", tokens));
      pp = dense(pool, at::kBFloat16, device, "kv_pool", 576 * slots);
    }
    const auto* tp = static_cast<const uint64_t*>(dense(&turns, at::kLong, device, "turns"));
    const auto* at_ = static_cast<const int64_t*>(dense(&positions, at::kLong, device, "positions"));
    const auto* np = static_cast<const int64_t*>(dense(valid, at::kLong, device, "num_valid"));
    const void* qwp = dense(qw, type, device, "q_weight", nope + rope_dim);
    const void* cwp = dense(cw, type, device, "c_weight", 512);
    uint32_t* err = static_cast<uint32_t*>(dense(tensor(a[15], "err"), at::kInt, device, "err"));
    const float eps = real(a[2]), amplitude = real(a[4]);
    const int layout = narrow(a[3]);
    void* stream = stream_of(a[16]);
    if (rope_dim > INT32_MAX || heads > INT32_MAX || nope > INT32_MAX) return MTV_E_BAD_ARGUMENT;
    const Unlocked unlocked;
    return norm_rope_write_entry(tp, int(rope_dim), amplitude, layout, at_, tokens, np, code, eps, vq.at, vq.tok, vq.head,
                               int(heads), int(nope), qwp, vn.at, vn.tok, vn.head, vr.at, vr.tok, vr.head, vc.at, vc.tok, cwp,
                               vk.at, vk.tok, lp, pp, slots, err, stream);
  });
}

// The addresses of mla_head_product, mla_prefill_run and mla_norm_rope_write; called once, before the others.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 3, [](PyObject* const* a) -> int {
    void* at[3];
    for (int i = 0; i < 3; ++i)
      if (!(at[i] = PyLong_AsVoidPtr(a[i]))) refuse(PyExc_ValueError, "an entry has no address");
    head_product_entry = reinterpret_cast<decltype(head_product_entry)>(at[0]);
    prefill_run_entry = reinterpret_cast<decltype(prefill_run_entry)>(at[1]);
    norm_rope_write_entry = reinterpret_cast<decltype(norm_rope_write_entry)>(at[2]);
    return 0;
  });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"head_product", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(head_product)), METH_FASTCALL, nullptr},
    {"prefill_run", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill_run)), METH_FASTCALL, nullptr},
    {"norm_rope_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm_rope_write)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "binding_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_binding_ext() { return PyModule_Create(&module); }
