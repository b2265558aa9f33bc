// The quick way from Python into the library for calls that the device answers in a few microseconds: one function a call that
// reads its tensors where they are (type, device, layout, size, address, stream) and calls the C entry.  pq.py goes through it
// when a call leaves every optional size to its tensors.  A call that is not plainly right returns -1 and has had no effect:
// pq.py then checks it argument by argument and says what is wrong.  One token through a 4096 x 4096 linear: 4 us on the host
// less than by attribute lookups and ctypes, whose 9 were more than the device's 7.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cxxabi.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/pq.h"

namespace {

// The library's entries, by their addresses in the copy that pq.py has loaded.
decltype(&pq_quant_fp4) quant_fp4 = nullptr;
decltype(&pq_fp4_gemm) fp4_gemm = nullptr;
decltype(&pq_fp4_linear) fp4_linear = nullptr;
decltype(&pq_kv4_attention_masked) attention_masked = nullptr;

PyObject* not_taken() {
  PyErr_Clear();
  return PyLong_FromLong(-1);
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A tensor of the current device and of this type, with memory and strides (sparse ones have none).
bool here(const at::Tensor* x, at::ScalarType type, int dev) {
  return x && x->defined() && x->layout() == at::kStrided && x->is_cuda() && x->get_device() == dev && x->scalar_type() == type;
}

// A dense one of at least `need` elements.
void* dense(PyObject* o, at::ScalarType type, int64_t need, int dev) {
  const at::Tensor* x = tensor(o);
  return here(x, type, dev) && x->is_contiguous() && x->numel() >= need ? x->data_ptr() : nullptr;
}

bool integer(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}

bool int32(PyObject* o, int64_t* v) { return integer(o, v) && *v == (int32_t)*v; }

bool number(PyObject* o, double* v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;   // no tensor: reading one would wait for the device
  *v = PyFloat_AsDouble(o);
  return !(*v == -1.0 && PyErr_Occurred());
}

bool format_of(PyObject* o, pq_fp4_format* f) {
  if (!PyUnicode_Check(o)) return false;
  if (PyUnicode_CompareWithASCIIString(o, "nv") == 0) *f = PQ_FP4_NV;
  else if (PyUnicode_CompareWithASCIIString(o, "mx") == 0) *f = PQ_FP4_MX;
  else return false;
  return true;
}

int64_t scale_bytes(int64_t rows, int64_t D, pq_fp4_format f) {
  const int64_t span = f == PQ_FP4_NV ? 64 : 128;
  return (rows + 127) / 128 * ((D + span - 1) / span) * 512;
}

// bf16 rows with a stride between them; a single row's stride says nothing.
struct Rows {
  void* p = nullptr;
  int64_t T = 0, D = 0, ld = 0;
};
bool rows_of(PyObject* o, int dev, Rows* r) {
  const at::Tensor* x = tensor(o);
  if (!here(x, at::kBFloat16, dev)) return false;
  if (x->dim() == 2) {
    if (x->stride(1) != 1) return false;
    r->D = x->size(1);
  } else if (x->dim() == 3) {                            // [T][heads][head_dim], the heads dense
    if (x->stride(2) != 1 || (x->stride(1) != x->size(2) && x->size(1) != 1)) return false;
    r->D = x->size(1) * x->size(2);
  } else {
    return false;
  }
  r->T = x->size(0);
  r->ld = r->T > 1 ? x->stride(0) : r->D;
  r->p = x->data_ptr();
  return true;
}

int device() {
  const int dev = c10::cuda::device_count() > 0 ? (int)c10::cuda::current_device() : -1;
  return dev;
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// Tensors without memory (fake ones, functional ones) throw when asked for it, and no exception may leave a C entry.  What
// unwinds a thread that ends (a daemon thread that asks for the lock after the interpreter's end) is none and goes on.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (abi::__forced_unwind&) {
    throw;
  } catch (...) {
    return not_taken();
  }
}

// The library's entry without the interpreter's lock.  What it throws ends here, where the lock can be taken again, and becomes
// Python's: the call may have had its effect, so it is not one that was not taken.
template <typename F>
PyObject* call(F f) {
  pq_status st = PQ_OK;
  bool threw = false;
  Py_BEGIN_ALLOW_THREADS
  try {
    st = f();
  } catch (abi::__forced_unwind&) {
    throw;
  } catch (...) {
    threw = true;
  }
  Py_END_ALLOW_THREADS
  if (threw) {
    PyErr_SetString(PyExc_RuntimeError, "the library ended with a C++ exception; whether the call was made is not known");
    return nullptr;
  }
  return PyLong_FromLong((long)st);
}

// quant_fp4(X, codes, scales, fmt, g, factor)
PyObject* py_quant_fp4(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return not_taken();
  const int dev = device();
  Rows X;
  pq_fp4_format f;
  int64_t g;
  double factor;
  if (dev < 0 || !rows_of(a[0], dev, &X) || tensor(a[0])->dim() != 2 || !format_of(a[3], &f) || !int32(a[4], &g) ||
      !number(a[5], &factor))
    return not_taken();
  void* codes = dense(a[1], at::kByte, X.T * X.D / 2, dev);
  void* scales = dense(a[2], at::kByte, scale_bytes(X.T, X.D, f), dev);
  if (!codes || !scales) return not_taken();
  void* stream = stream_of(dev);
  return call([&] {
    return quant_fp4(X.p, X.T, X.D, X.ld, (int)g, f, (float)factor, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), stream);
  });
}

struct Product {
  void *ca, *sa, *cw, *sw, *Y;
  int64_t N;
  pq_out_dtype out;
};
// codes_A, scales_A, codes_W, scales_W and Y at a[0..4].
bool product(PyObject* const* a, int64_t T, int64_t D, pq_fp4_format f, int dev, Product* p) {
  const at::Tensor *w = tensor(a[2]), *y = tensor(a[4]);
  if (!w || !w->defined() || w->dim() < 1 || !y || !y->defined()) return false;
  if (w->dim() == 2 && w->size(1) != D / 2) return false;
  if (y->scalar_type() != at::kBFloat16 && y->scalar_type() != at::kFloat) return false;
  p->N = w->size(0);
  p->out = y->scalar_type() == at::kBFloat16 ? PQ_OUT_BF16 : PQ_OUT_F32;
  p->ca = dense(a[0], at::kByte, T * (D / 2), dev);
  p->sa = dense(a[1], at::kByte, scale_bytes(T, D, f), dev);
  p->cw = dense(a[2], at::kByte, p->N * (D / 2), dev);
  p->sw = dense(a[3], at::kByte, scale_bytes(p->N, D, f), dev);
  p->Y = dense(a[4], y->scalar_type(), T * p->N, dev);
  return p->ca && p->sa && p->cw && p->sw && p->Y;
}

// fp4_gemm(codes_A, scales_A, codes_W, scales_W, Y, fmt, alpha)
PyObject* py_fp4_gemm(PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return not_taken();
  const int dev = device();
  pq_fp4_format f;
  double alpha;
  Product p;
  const at::Tensor* ca = tensor(a[0]);
  if (dev < 0 || !ca || !ca->defined() || ca->dim() != 2 || !format_of(a[5], &f) || !number(a[6], &alpha)) return not_taken();
  const int64_t T = ca->size(0), D = 2 * ca->size(1);
  if (!product(a, T, D, f, dev, &p)) return not_taken();
  void* stream = stream_of(dev);
  return call([&] {
    return fp4_gemm(static_cast<const uint8_t*>(p.ca), static_cast<const uint8_t*>(p.sa), static_cast<const uint8_t*>(p.cw),
                    static_cast<const uint8_t*>(p.sw), T, p.N, D, f, (float)alpha, p.Y, p.out, stream);
  });
}

// fp4_linear(X, codes_A, scales_A, codes_W, scales_W, Y, fmt, g, factor_A, factor_W)
PyObject* py_fp4_linear(PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return not_taken();
  const int dev = device();
  Rows X;
  pq_fp4_format f;
  int64_t g;
  double fa, fw;
  Product p;
  if (dev < 0 || !rows_of(a[0], dev, &X) || tensor(a[0])->dim() != 2 || !format_of(a[6], &f) || !int32(a[7], &g) ||
      !number(a[8], &fa) || !number(a[9], &fw) || !product(a + 1, X.T, X.D, f, dev, &p))
    return not_taken();
  void* stream = stream_of(dev);
  return call([&] {
    return fp4_linear(X.p, X.T, X.D, X.ld, (int)g, f, (float)fa, static_cast<uint8_t*>(p.ca), static_cast<uint8_t*>(p.sa),
                      static_cast<const uint8_t*>(p.cw), static_cast<const uint8_t*>(p.sw), (float)fw, p.N, p.Y, p.out, stream);
  });
}

// attention_masked(cache handle, cache device, Q, O, q_start, seq_lens, block_table, max_q, max_len, scale, window, sinks, tree)
PyObject* py_attention_masked(PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return not_taken();
  const int dev = device();
  int64_t handle, on, max_q, max_len, window, sinks;
  if (dev < 0 || !integer(a[0], &handle) || !integer(a[1], &on) || on != dev || !integer(a[7], &max_q) || !integer(a[8], &max_len) ||
      !integer(a[10], &window) || !integer(a[11], &sinks))
    return not_taken();
  const pq_kv4_cache* cache = reinterpret_cast<const pq_kv4_cache*>((uintptr_t)handle);
  const int64_t hd = cache->head_dim;
  double scale = std::pow((double)hd, -0.5);
  Rows Q, O;
  if ((a[9] != Py_None && !number(a[9], &scale)) || !rows_of(a[2], dev, &Q) || !rows_of(a[3], dev, &O) || Q.D != O.D || Q.T != O.T ||
      hd <= 0 || Q.D % hd != 0)
    return not_taken();
  const at::Tensor* table = tensor(a[6]);
  if (!table || !table->defined() || table->dim() != 2) return not_taken();
  const int64_t B = table->size(0), width = table->size(1);
  void *starts = dense(a[4], at::kInt, B + 1, dev), *lens = dense(a[5], at::kInt, B, dev), *pages = dense(a[6], at::kInt, B * width, dev);
  void* lists = nullptr;
  int64_t words = 0;
  if (a[12] != Py_None) {
    const at::Tensor* tree = tensor(a[12]);
    if (!tree || !tree->defined() || tree->dim() != 2 || tree->size(0) != Q.T) return not_taken();
    words = tree->size(1);
    lists = dense(a[12], at::kInt, Q.T * words, dev);
    if (!lists) return not_taken();
  }
  if (!starts || !lens || !pages) return not_taken();
  void* stream = stream_of(dev);
  return call([&] {
    return attention_masked(cache, Q.p, Q.ld, (int)(Q.D / hd), static_cast<const int32_t*>(starts), static_cast<const int32_t*>(lens),
                            static_cast<const int32_t*>(pages), width, B, Q.T, max_q, max_len, (float)scale, window, sinks,
                            static_cast<const uint32_t*>(lists), words, O.p, O.ld, stream);
  });
}

// bind(addresses of pq_quant_fp4, pq_fp4_gemm, pq_fp4_linear, pq_kv4_attention_masked)
PyObject* py_bind(PyObject* const* a, Py_ssize_t n) {
  int64_t v[4];
  for (Py_ssize_t i = 0; i < 4; ++i)
    if (n != 4 || !integer(a[i], &v[i])) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind: expected four addresses");
      return nullptr;
    }
  quant_fp4 = reinterpret_cast<decltype(quant_fp4)>((uintptr_t)v[0]);
  fp4_gemm = reinterpret_cast<decltype(fp4_gemm)>((uintptr_t)v[1]);
  fp4_linear = reinterpret_cast<decltype(fp4_linear)>((uintptr_t)v[2]);
  attention_masked = reinterpret_cast<decltype(attention_masked)>((uintptr_t)v[3]);
  Py_RETURN_NONE;
}

#define PQ_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<py_##name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PQ_METHOD(bind), PQ_METHOD(quant_fp4), PQ_METHOD(fp4_gemm), PQ_METHOD(fp4_linear),
                         PQ_METHOD(attention_masked), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pqcall", "Calls of libpq with tensors read in place.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pqcall() { return PyModule_Create(&module); }
