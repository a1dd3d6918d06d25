// Argument checks and marshalling of the short calls, in C++.
//
// A decode step's norm, cache write and attention over a short cache take the
// GPU 3 to 13 us; the same checks in Python, with a ctypes call of 25
// arguments, took the host 7 to 8 us on top of the launch. Each function here
// checks its tensors as the Python wrappers of the other entry points do
// (ValueError), calls the C ABI entry point of the same name and returns its
// status. No arithmetic, no allocation, no state.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "tq.h"

namespace {

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
void need(bool ok, const char* text) {
  if (!ok) throw Bad(text);
}

// A tensor argument, or NULL for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& must(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw Bad(std::string(name) + " is None");
  return *t;
}
void* at_(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

int on_device(std::initializer_list<const at::Tensor*> all) {
  int dev = -1;
  for (const at::Tensor* t : all) {
    if (!t) continue;
    const int d = t->is_cuda() ? t->get_device() : -1;
    if (dev < 0) dev = d;
    need(d >= 0 && d == dev, "all tensors must be CUDA tensors on one device");
  }
  need(dev == c10::cuda::current_device(), "the tensors must be on the current device");
  return dev;
}

const int32_t* int32s(const at::Tensor* t, const char* name, std::initializer_list<int64_t> shape) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || !t->is_contiguous() || t->sizes() != at::IntArrayRef(shape))
    throw Bad(std::string(name) + " must be a contiguous int32 tensor of the documented shape");
  return static_cast<const int32_t*>(t->data_ptr());
}
int32_t* status_word(const at::Tensor* t) {
  if (!t) return nullptr;
  need(t->scalar_type() == at::kInt && t->numel() > 0, "d_status must be an int32 tensor with an element");
  return static_cast<int32_t*>(t->data_ptr());
}
tq_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return TQ_F32;
  need(t.scalar_type() == at::kBFloat16, "unsupported dtype (float32 or bfloat16)");
  return TQ_BF16;
}
// Unit stride along d (a tensor without elements has no strides that matter).
void rows(const at::Tensor& t, const char* text) { need(t.numel() == 0 || t.stride(-1) == 1, text); }

void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw Bad("stream must be a torch.cuda.Stream, an integer handle or None");
  return p;
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Bad("a number was expected");
  return x;
}
int64_t whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Bad("a whole number was expected");
  return x;
}
int32_t whole32(PyObject* o) {
  const int64_t x = whole(o);
  need(x >= INT32_MIN && x <= INT32_MAX, "a 32-bit whole number was expected");
  return static_cast<int32_t>(x);
}
int32_t size32(int64_t x) {
  need(x <= INT32_MAX, "a tensor has 2^31 or more of something");
  return static_cast<int32_t>(x);
}

// k, v, k_scale, v_scale, code: the five fields of a Cache8.
tq_cache8 cache_of(PyObject* const* o, const at::Tensor* (&t)[4]) {
  static const char* const names[4] = {"cache.k", "cache.v", "cache.k_scale", "cache.v_scale"};
  for (int i = 0; i < 4; ++i) t[i] = &must(o[i], names[i]);
  need(t[0]->dim() == 4 && t[1]->sizes() == t[0]->sizes(), "a Cache8 has [n_blocks, heads, block, d] codes");
  for (int i = 0; i < 4; ++i) {
    need(t[i]->is_contiguous() && t[i]->scalar_type() == (i < 2 ? at::kByte : at::kFloat),
         "a Cache8 has contiguous uint8 codes and float32 scales");
    if (i >= 2)
      need(t[i]->dim() == 2 && t[i]->size(0) == t[0]->size(0) && t[i]->size(1) == t[0]->size(1),
           "a Cache8 has [n_blocks, heads] scales");
  }
  const char* code = PyUnicode_Check(o[4]) ? PyUnicode_AsUTF8(o[4]) : nullptr;
  const std::string c = code ? code : "";
  need(c == "e4m3" || c == "int8", "unknown code (e4m3 or int8)");
  tq_cache8 r{};
  r.d = size32(t[0]->size(3));
  r.heads = size32(t[0]->size(1));
  r.block = size32(t[0]->size(2));
  r.code = c == "e4m3" ? TQ_E4M3 : TQ_INT8;
  r.n_blocks = t[0]->size(0);
  r.k = static_cast<uint8_t*>(t[0]->data_ptr());
  r.v = static_cast<uint8_t*>(t[1]->data_ptr());
  r.k_scale = static_cast<float*>(t[2]->data_ptr());
  r.v_scale = static_cast<float*>(t[3]->data_ptr());
  return r;
}
// A block table and its stride (without one, every sequence has an equal share of the pages).
const int32_t* table_of(const at::Tensor* t, const tq_cache8& c, int64_t batch, int64_t* stride) {
  if (!t) {
    *stride = c.n_blocks / (batch > 0 ? batch : 1);
    return nullptr;
  }
  need(t->dim() == 2 && t->size(0) == batch && t->scalar_type() == at::kInt && t->is_contiguous(),
       "block_table must be a contiguous int32 [batch, blocks] tensor");
  *stride = t->size(1);
  return static_cast<const int32_t*>(t->data_ptr());
}

PyObject* status(tq_status s) { return PyLong_FromLong(static_cast<long>(s)); }

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_Clear();
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// q, k, q_out, k_out, q_weight, k_weight, eps, positions, rope_base, rot_dim, d_status, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor* x[4] = {tensor(a[0], "q"), tensor(a[1], "k"), tensor(a[2], "q_out"), tensor(a[3], "k_out")};
    need(!x[0] == !x[2] && !x[1] == !x[3], "q and q_out, and k and k_out, go together");
    const at::Tensor* one = x[0] ? x[0] : x[1];
    need(one && one->dim() == 3, "q and k must be [tokens, heads, d] tensors, one of them at least");
    const int64_t tokens = one->size(0), d = one->size(2);
    int64_t ts[4] = {}, hs[4] = {};
    for (int i = 0; i < 4; ++i) {
      if (!x[i]) continue;
      need(x[i]->dim() == 3 && x[i]->size(0) == tokens && x[i]->size(2) == d && x[i]->sizes() == x[i & 1]->sizes(),
           "q, k and their outputs must be [tokens, heads, d] tensors, an output as its input");
      rows(*x[i], "q, k and their outputs must have unit stride along d");
      need(x[i]->scalar_type() == one->scalar_type(), "q, k and their outputs must have one dtype");
      ts[i] = x[i]->stride(0);
      hs[i] = x[i]->stride(1);
    }
    const at::Tensor* w[2] = {tensor(a[4], "q_weight"), tensor(a[5], "k_weight")};
    for (const at::Tensor* y : w)
      need(!y || (y->scalar_type() == at::kFloat && y->is_contiguous() && y->dim() == 1 && y->size(0) == d),
           "weights must be contiguous float32 tensors of shape [d]");
    const at::Tensor *pos = tensor(a[7], "positions"), *st = tensor(a[10], "d_status");
    const int dev = on_device({x[0], x[1], x[2], x[3], w[0], w[1], pos, st});
    return status(tq_qk_norm_rope(size32(d), a[9] == Py_None ? size32(d) : whole32(a[9]), tokens,
                                  x[0] ? size32(x[0]->size(1)) : 0, x[1] ? size32(x[1]->size(1)) : 0, dtype_of(*one),
                                  at_(x[0]), ts[0], hs[0], at_(x[1]), ts[1], hs[1], at_(x[2]), ts[2], hs[2], at_(x[3]),
                                  ts[3], hs[3], static_cast<const float*>(at_(w[0])), static_cast<const float*>(at_(w[1])),
                                  static_cast<float>(number(a[6])), int32s(pos, "positions", {tokens}),
                                  static_cast<float>(number(a[8])), status_word(st), stream_of(a[11], dev)));
  });
}

// write, cache (5), k, v, cu_tokens, start, block_table, d_status, stream
PyObject* cache8_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const bool write = a[0] == Py_True;
    const at::Tensor* t[4];
    const tq_cache8 c = cache_of(a + 1, t);
    const at::Tensor *k = tensor(a[6], "k"), *v = tensor(a[7], "v");
    need(write ? k && v : k || v, write ? "k and v are needed" : "k_out and v_out are both None");
    const at::Tensor& one = k ? *k : *v;
    for (const at::Tensor* x : {k, v}) {
      if (!x) continue;
      need(x->dim() == 3 && x->size(0) == one.size(0) && x->size(1) == c.heads && x->size(2) == c.d &&
               x->scalar_type() == one.scalar_type(),
           "k and v must be [tokens, heads, d] tensors of one dtype with the cache's heads and d");
      rows(*x, "k and v must have unit stride along d");
    }
    const at::Tensor &cu = must(a[8], "cu_tokens"), &start = must(a[9], "start");
    need(start.dim() == 1, "start must be an int32 [batch] tensor");
    const int64_t batch = start.size(0);
    const at::Tensor *table = tensor(a[10], "block_table"), *st = tensor(a[11], "d_status");
    const int dev = on_device({t[0], t[1], t[2], t[3], k, v, &cu, &start, table, st});
    int64_t stride = 0;
    const int32_t* tp = table_of(table, c, batch, &stride);
    const int32_t *cp = int32s(&cu, "cu_tokens", {batch + 1}), *sp = int32s(&start, "start", {batch});
    const int64_t kt = k ? k->stride(0) : 0, kh = k ? k->stride(1) : 0, vt = v ? v->stride(0) : 0, vh = v ? v->stride(1) : 0;
    void* s = stream_of(a[12], dev);
    if (write)
      return status(tq_cache8_write(&c, dtype_of(one), at_(k), kt, kh, at_(v), vt, vh, one.size(0), size32(batch), cp, sp, tp,
                                    stride, status_word(st), s));
    return status(tq_cache8_read(&c, dtype_of(one), at_(k), kt, kh, at_(v), vt, vh, one.size(0), size32(batch), cp, sp, tp,
                                 stride, status_word(st), s));
  });
}

// cache (5), q, seq_lens, out, workspace, block_table, causal, window, scale, lse_out, d_status, stream
PyObject* cache8_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor* t[4];
    const tq_cache8 c = cache_of(a, t);
    const at::Tensor &q = must(a[5], "q"), &lens = must(a[6], "seq_lens"), &out = must(a[7], "out"), &ws = must(a[8], "workspace");
    need(q.dim() == 4 && out.sizes() == q.sizes(), "q and out must be [batch, hq, nq, d] tensors of the same shape");
    rows(q, "q must have unit stride along d");
    rows(out, "out must have unit stride along d");
    need(q.size(3) == c.d, "q's d is not the cache's");
    const int64_t batch = q.size(0), hq = q.size(1), nq = q.size(2);
    const at::Tensor *table = tensor(a[9], "block_table"), *lse = tensor(a[13], "lse_out"), *st = tensor(a[14], "d_status");
    need(!lse || (lse->scalar_type() == at::kFloat && lse->is_contiguous() && lse->dim() == 3 && lse->size(0) == batch &&
                  lse->size(1) == hq && lse->size(2) == nq),
         "lse_out must be a contiguous float32 [batch, hq, nq] tensor");
    need(ws.is_contiguous(), "workspace must be contiguous");
    const int dev = on_device({t[0], t[1], t[2], t[3], &q, &lens, &out, &ws, table, lse, st});
    int64_t stride = 0;
    const int32_t* tp = table_of(table, c, batch, &stride);
    const int causal = PyObject_IsTrue(a[10]);
    if (causal < 0) throw Bad("causal must be a truth value");
    const double scale = a[12] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : number(a[12]);
    return status(tq_cache8_attention(&c, q.data_ptr(), dtype_of(q), q.stride(0), q.stride(1), q.stride(2), size32(batch),
                                      size32(hq), size32(nq), int32s(&lens, "seq_lens", {batch}), tp, stride, causal,
                                      whole32(a[11]), static_cast<float>(scale), out.data_ptr(), dtype_of(out), out.stride(0),
                                      out.stride(1), out.stride(2), static_cast<float*>(at_(lse)), ws.data_ptr(), ws.nbytes(),
                                      status_word(st), stream_of(a[15], dev)));
  });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"cache8_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache8_rows)), METH_FASTCALL, nullptr},
    {"cache8_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache8_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tq_torch", "Checks and marshalling of libtq.so's short calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tq_torch(void) { return PyModule_Create(&module); }
