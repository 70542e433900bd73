// Native front of the serving operators for the binding: single-token calls take a few microseconds on the
// GPU, less than the Python checks, allocations and argument conversion of a ctypes call.  Each function
// looks at its tensors, allocates the outputs and makes the C-ABI call; where anything is not the plain case
// it returns None, and the Python wrapper, which says what is wrong, takes over.  A status that is not
// GPTQ_OK is returned as a number.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <cmath>

#include "../../include/gptq.h"

namespace {

decltype(&gptq_rotary) p_rotary = nullptr;
decltype(&gptq_cache_write) p_write = nullptr;
decltype(&gptq_cache_read) p_read = nullptr;
decltype(&gptq_paged_attention) p_attention = nullptr;

using at::Tensor;

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int code(at::ScalarType t) { return t == at::kHalf ? GPTQ_F16 : t == at::kBFloat16 ? GPTQ_BF16 : -1; }

// [tokens, heads, head_dim], unit stride inside a head, on device `dev`
bool heads(const Tensor* t, at::ScalarType type, int dev) {
  return t && t->dim() == 3 && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->stride(2) == 1 &&
         !t->requires_grad();
}
bool plain(const Tensor* t, at::ScalarType type, int dev, c10::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape && t->is_contiguous();
}
int64_t stride(const Tensor* t, int d) { return t->size(d) > 1 ? t->stride(d) : 0; }

// A small whole number; false for anything else, without an exception.
bool whole(PyObject* o, long* v) {
  if (!PyLong_Check(o)) return false;
  int past = 0;
  *v = PyLong_AsLongAndOverflow(o, &past);
  return past == 0;
}

struct Cache {
  void *k, *v;
  float *ks, *vs;
  uint8_t *kz, *vz;
  int64_t pages, heads, page, dim;
  int bits;
};

// o: k, v, k_scales, k_zeros, v_scales, v_zeros (the last four None at 16 bits)
bool cache(PyObject* const* o, long bits, int dev, Cache* c, at::ScalarType* type) {
  const Tensor *k = tensor(o[0]), *v = tensor(o[1]);
  if (!k || !v || k->dim() != 4 || (bits != 16 && bits != 8 && bits != 4)) return false;
  *type = k->scalar_type();
  if (bits == 16 ? code(*type) < 0 : *type != at::kByte) return false;
  if (!plain(k, *type, dev, k->sizes()) || !plain(v, *type, dev, k->sizes())) return false;
  *c = Cache{k->data_ptr(), v->data_ptr(), nullptr, nullptr, nullptr, nullptr, k->size(0), k->size(1), k->size(2),
             k->size(3) * (bits == 4 ? 2 : 1), static_cast<int>(bits)};
  if (bits < 16) {
    const Tensor *ks = tensor(o[2]), *kz = tensor(o[3]), *vs = tensor(o[4]), *vz = tensor(o[5]);
    const auto shape = k->sizes().slice(0, 3);
    if (!plain(ks, at::kFloat, dev, shape) || !plain(kz, at::kByte, dev, shape) || !plain(vs, at::kFloat, dev, shape) ||
        !plain(vz, at::kByte, dev, shape))
      return false;
    c->ks = static_cast<float*>(ks->data_ptr());
    c->kz = static_cast<uint8_t*>(kz->data_ptr());
    c->vs = static_cast<float*>(vs->data_ptr());
    c->vz = static_cast<uint8_t*>(vz->data_ptr());
  }
  return true;
}

PyObject* none() { Py_RETURN_NONE; }
void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

// The library's calls (an allocation from its pool, up to four launches) run without the interpreter's lock, as
// calls through ctypes do: threads that serve at once do not take turns.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
int unlocked(F* f, A... a) {
  Unlocked u;
  return f(a...);
}

#define GUARD_BEGIN try {
#define GUARD_END                                     \
  }                                                   \
  catch (const std::exception& e) {                   \
    PyErr_SetString(PyExc_RuntimeError, e.what());    \
    return nullptr;                                   \
  }

// rotary(q, k or None, positions, inv_freq, attention_factor, interleaved)
PyObject* rotary(PyObject*, PyObject* const* o, Py_ssize_t n) {
  GUARD_BEGIN
  if (n != 6 || !p_rotary) return none();
  const Tensor *q = tensor(o[0]), *k = tensor(o[1]), *pos = tensor(o[2]), *f = tensor(o[3]);
  if (!q || (!k && o[1] != Py_None) || !f || !q->is_cuda() || code(q->scalar_type()) < 0) return none();
  const int dev = q->get_device();
  if (dev != c10::cuda::current_device() || !heads(q, q->scalar_type(), dev)) return none();
  const int64_t T = q->size(0), H = q->size(1), D = q->size(2), HK = k ? k->size(1) : 0;
  if (k && (!heads(k, q->scalar_type(), dev) || k->size(0) != T || k->size(2) != D)) return none();
  if (!plain(pos, at::kInt, dev, {T}) || f->dim() != 1 || !plain(f, at::kDouble, dev, f->sizes())) return none();
  const double factor = PyFloat_AsDouble(o[4]);
  const int inter = PyObject_IsTrue(o[5]);
  if (PyErr_Occurred() || inter < 0) {
    PyErr_Clear();
    return none();
  }
  Tensor qo = at::empty({T, H, D}, q->options()), ko;
  if (k) ko = at::empty({T, HK, D}, q->options());
  const int st = unlocked(p_rotary, q->data_ptr(), k ? k->data_ptr() : nullptr, code(q->scalar_type()), T,
                          static_cast<int>(H), static_cast<int>(HK), static_cast<int>(D),
                          static_cast<int>(2 * f->size(0)), inter, stride(q, 0), stride(q, 1),
                          k ? stride(k, 0) : 0, k ? stride(k, 1) : 0,
                          static_cast<const int32_t*>(pos->data_ptr()), static_cast<const double*>(f->data_ptr()),
                          static_cast<float>(factor), qo.data_ptr(), k ? ko.data_ptr() : nullptr, H * D, D, HK * D, D,
                          stream(dev));
  if (st != GPTQ_OK) return PyLong_FromLong(st);
  if (k) return pair(qo, ko);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(qo));
  PyTuple_SET_ITEM(r, 1, Py_NewRef(Py_None));
  return r;
  GUARD_END
}

// cache_write(k, v, cache's six, slots, bits) -> True
PyObject* cache_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  GUARD_BEGIN
  long bits;
  if (n != 10 || !p_write || !whole(o[9], &bits)) return none();
  const Tensor *k = tensor(o[0]), *v = tensor(o[1]), *slots = tensor(o[8]);
  if (!k || !k->is_cuda() || code(k->scalar_type()) < 0) return none();
  const int dev = k->get_device();
  if (dev != c10::cuda::current_device() || !heads(k, k->scalar_type(), dev) || !heads(v, k->scalar_type(), dev) ||
      v->sizes() != k->sizes())
    return none();
  Cache c;
  at::ScalarType type;
  if (!cache(o + 2, bits, dev, &c, &type) || c.heads != k->size(1) || c.dim != k->size(2) ||
      (bits == 16 && type != k->scalar_type()) || !plain(slots, at::kInt, dev, {k->size(0)}))
    return none();
  const int st = unlocked(p_write, k->data_ptr(), v->data_ptr(), code(k->scalar_type()), k->size(0),
                          static_cast<int>(c.heads), static_cast<int>(c.dim), stride(k, 0), stride(k, 1), stride(v, 0),
                          stride(v, 1), c.k, c.v, c.ks, c.kz, c.vs, c.vz, c.bits, c.pages, static_cast<int>(c.page),
                          static_cast<const int32_t*>(slots->data_ptr()), stream(dev));
  if (st != GPTQ_OK) return PyLong_FromLong(st);
  Py_RETURN_TRUE;
  GUARD_END
}

// cache_read(cache's six, slots, bits, half) -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* o, Py_ssize_t n) {
  GUARD_BEGIN
  long bits;
  if (n != 9 || !p_read || !whole(o[7], &bits)) return none();
  const Tensor* slots = tensor(o[6]);
  if (!slots || !slots->is_cuda() || slots->dim() != 1) return none();
  const int dev = slots->get_device();
  const at::ScalarType type = o[8] == Py_True ? at::kHalf : at::kBFloat16;
  Cache c;
  at::ScalarType held;
  if (dev != c10::cuda::current_device() || !plain(slots, at::kInt, dev, slots->sizes()) ||
      !cache(o, bits, dev, &c, &held) || (bits == 16 && held != type))
    return none();
  const int64_t count = slots->size(0);
  const auto opt = slots->options().dtype(type);
  Tensor k = at::empty({count, c.heads, c.dim}, opt), v = at::empty({count, c.heads, c.dim}, opt);
  const int st = unlocked(p_read, c.k, c.v, c.ks, c.kz, c.vs, c.vz, c.bits, c.pages, static_cast<int>(c.page),
                          static_cast<const int32_t*>(slots->data_ptr()), count, static_cast<int>(c.heads),
                          static_cast<int>(c.dim), code(type), k.data_ptr(), v.data_ptr(), stream(dev));
  if (st != GPTQ_OK) return PyLong_FromLong(st);
  return pair(k, v);
  GUARD_END
}

// paged_attention(q, cache's six, table, lens, starts, bits, max_q or None, causal, scale or None) -> out
PyObject* paged_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
  GUARD_BEGIN
  long bits, rows = 0;
  if (n != 14 || !p_attention || !whole(o[10], &bits) || (o[11] != Py_None && (!whole(o[11], &rows) || rows < 0)))
    return none();
  const Tensor *q = tensor(o[0]), *table = tensor(o[7]), *lens = tensor(o[8]), *starts = tensor(o[9]);
  if (!q || !q->is_cuda() || code(q->scalar_type()) < 0 || !table || table->dim() != 2) return none();
  const int dev = q->get_device();
  Cache c;
  at::ScalarType held;
  if (dev != c10::cuda::current_device() || !heads(q, q->scalar_type(), dev) || !cache(o + 1, bits, dev, &c, &held) ||
      (bits == 16 && held != q->scalar_type()) || c.dim != q->size(2) || !c.heads || q->size(1) % c.heads)
    return none();
  const int64_t T = q->size(0), H = q->size(1), S = table->size(0);
  if (!plain(table, at::kInt, dev, table->sizes()) || !plain(lens, at::kInt, dev, {S}) || !plain(starts, at::kInt, dev, {S + 1}))
    return none();
  const int64_t most = o[11] == Py_None ? T : rows;
  const int causal = PyObject_IsTrue(o[12]);
  const double scale = o[13] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.dim)) : PyFloat_AsDouble(o[13]);
  if (causal < 0 || PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  Tensor out = at::empty({T, H, c.dim}, q->options());
  const int st = unlocked(p_attention, q->data_ptr(), code(q->scalar_type()), T, static_cast<int>(H),
                          static_cast<int>(c.heads), static_cast<int>(c.dim), stride(q, 0), stride(q, 1), c.k, c.v, c.ks,
                          c.kz, c.vs, c.vz, c.bits, c.pages, static_cast<int>(c.page),
                          static_cast<const int32_t*>(table->data_ptr()),
                          table->size(1), static_cast<const int32_t*>(lens->data_ptr()),
                          static_cast<const int32_t*>(starts->data_ptr()), S, most, causal, static_cast<float>(scale),
                          out.data_ptr(), stream(dev));
  if (st != GPTQ_OK) return PyLong_FromLong(st);
  return THPVariable_Wrap(out);
  GUARD_END
}

// open(path of the native library): its functions
PyObject* open_library(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  p_rotary = reinterpret_cast<decltype(p_rotary)>(dlsym(h, "gptq_rotary"));
  p_write = reinterpret_cast<decltype(p_write)>(dlsym(h, "gptq_cache_write"));
  p_read = reinterpret_cast<decltype(p_read)>(dlsym(h, "gptq_cache_read"));
  p_attention = reinterpret_cast<decltype(p_attention)>(dlsym(h, "gptq_paged_attention"));
  if (!p_rotary || !p_write || !p_read || !p_attention) {
    PyErr_SetString(PyExc_RuntimeError, "the native library lacks a serving operator");
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"open", open_library, METH_O, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_write)), METH_FASTCALL, nullptr},
    {"cache_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_read)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
