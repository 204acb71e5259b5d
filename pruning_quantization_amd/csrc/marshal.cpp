// Python marshalling of the calls that a serving step makes once per layer and
// token (int8_gemm, kv_append, kv_attention): checks of the tensors, the C
// descriptors, the outputs and the current stream, in native code because in
// Python they took as long as the kernels (9 to 15 us a call against 5 to 10).
// The C entry points themselves are handed in by bind(), as loaded by
// binding.py, which also holds the documentation and the defaults.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cmath>
#include <exception>
#include <sstream>
#include <string>
#include <vector>

#include "sparq24.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&sparq24_int8_gemm) c_int8_gemm = nullptr;
decltype(&sparq24_kv_append) c_kv_append = nullptr;
decltype(&sparq24_kv_attention) c_kv_attention = nullptr;

PyObject* call_error = nullptr;  // class raised for a status: (function, status)

struct PyError : std::exception {
  PyObject* type;
  std::string text;
  PyError(PyObject* t, std::string s) : type(t), text(std::move(s)) {}
};
[[noreturn]] void value_error(const std::string& s) { throw PyError(PyExc_ValueError, s); }
[[noreturn]] void type_error(const std::string& s) { throw PyError(PyExc_TypeError, s); }

std::string shape_of(const Tensor& t) {
  std::ostringstream o;
  o << t.sizes() << ' ' << t.scalar_type();
  return o.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int dtype_code(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return SPARQ24_F32;
    case ScalarType::BFloat16: return SPARQ24_BF16;
    case ScalarType::Half: return SPARQ24_F16;
    default: type_error(std::string("unsupported dtype ") + c10::toString(t));
  }
}

template <class T>
T* vector(const Tensor& t, int64_t n, ScalarType type, const char* name) {
  if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
    value_error(std::string(name) + " must be contiguous " + c10::toString(type) + " with " + std::to_string(n) +
                " elements, got " + shape_of(t));
  return (T*)t.data_ptr();
}

// All tensors on one GPU; its index.  Last of a call's checks.
int device_of(std::initializer_list<const Tensor*> ts) {
  const Tensor* first = *ts.begin();
  const auto d = first->device();
  for (const Tensor* t : ts)
    if (t && t->device() != d) value_error("tensors on " + d.str() + " and " + t->device().str());
  if (!d.is_cuda()) value_error("tensors must be on a GPU, got " + d.str());
  return d.index();
}

// Runs f(stream) with the device current and other Python threads free to run.
template <class F>
int on_device(int dev, F&& f) {
  struct Released {
    PyThreadState* s = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(s); }
  } released;
  struct Current {
    const c10::DeviceIndex was = c10::hip::current_device(), dev;
    explicit Current(int d) : dev((c10::DeviceIndex)d) {
      if (was != dev) c10::hip::set_device(dev);
    }
    ~Current() {
      if (was != dev) (void)hipSetDevice(was);  // no throw
    }
  } current(dev);
  return f((hipStream_t)c10::hip::getCurrentHIPStream(current.dev).stream());
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) type_error("wrong number of arguments");
}

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const PyError& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* failed(const char* fn, int st) {
  if (PyObject* e = PyObject_CallFunction(call_error, "si", fn, st)) {
    PyErr_SetObject(call_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// bind(address of sparq24_int8_gemm, of sparq24_kv_append, of sparq24_kv_attention, error class)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 4);
    c_int8_gemm = (decltype(c_int8_gemm))PyLong_AsVoidPtr(a[0]);
    c_kv_append = (decltype(c_kv_append))PyLong_AsVoidPtr(a[1]);
    c_kv_attention = (decltype(c_kv_attention))PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Py_XDECREF(call_error);
    call_error = Py_NewRef(a[3]);
    Py_RETURN_NONE;
  });
}

// int8_gemm(codes_a, scale_a, codes_b, scale_b, bias, dtype, out)
PyObject* py_int8_gemm(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    arguments(argc, 7);
    const Tensor &ca = tensor(a[0], "codes_a"), &sa = tensor(a[1], "scale_a");
    const Tensor &cb = tensor(a[2], "codes_b"), &sb = tensor(a[3], "scale_b");
    const Tensor *bias = optional(a[4], "bias"), *given = optional(a[6], "out");
    if (ca.scalar_type() != ScalarType::Char || cb.scalar_type() != ScalarType::Char)
      type_error("int8 codes expected, got " + shape_of(ca) + " and " + shape_of(cb));
    const int64_t rank = ca.dim();
    if (cb.dim() != 2 || rank < 1 || ca.size(-1) != cb.size(1))
      value_error("shapes " + shape_of(ca) + " and " + shape_of(cb) + " do not multiply");
    const int64_t n = cb.size(0), k = cb.size(1);
    int64_t m = 1;
    for (int64_t i = 0; i + 1 < rank; ++i) m *= ca.size(i);
    // Step between the m rows of t, whose leading dims have to be evenly spaced.
    auto rows = [&](const Tensor& t, int64_t width, const char* name) -> int64_t {
      if (m == 0) return width;
      if (width > 1 && t.stride(-1) != 1) value_error(std::string(name) + " must be contiguous along its last dim");
      bool one = true;
      int64_t step = width, span = 0;
      for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (one) span = step = t.stride(i);
        one = false;
        if (t.stride(i) != span) value_error("the rows of " + std::string(name) + " must be evenly spaced");
        span *= t.size(i);
      }
      return step;
    };
    const int64_t lda = rows(ca, k, "codes_a"), ldb = n > 1 ? cb.stride(0) : k;
    if (k > 1 && n && cb.stride(1) != 1) value_error("codes_b must be contiguous along K");
    if (!THPDtype_Check(a[5])) type_error("dtype must be a torch.dtype");
    const ScalarType want = given ? given->scalar_type() : ((THPDtype*)a[5])->scalar_type;
    const int code = dtype_code(want);
    float* psa = vector<float>(sa, m, ScalarType::Float, "scale_a");
    float* psb = vector<float>(sb, n, ScalarType::Float, "scale_b");
    float* pbias = bias ? vector<float>(*bias, n, ScalarType::Float, "bias") : nullptr;
    std::vector<int64_t> shape(ca.sizes().begin(), ca.sizes().end());
    shape.back() = n;
    if (given && given->sizes() != at::IntArrayRef(shape)) value_error("out has shape " + shape_of(*given));
    const int64_t ldc = given ? rows(*given, n, "out") : n;
    const int dev = device_of({&ca, &sa, &cb, &sb, bias, given});
    const Tensor out = given ? *given : at::empty(shape, ca.options().dtype(want));
    const int st = on_device(dev, [&](hipStream_t s) {
      return c_int8_gemm((const int8_t*)ca.data_ptr(), lda, psa, m, (const int8_t*)cb.data_ptr(), ldb, psb, n, k,
                         pbias, code, out.data_ptr(), ldc, nullptr, nullptr, s);
    });
    return st ? failed("sparq24_int8_gemm", st) : THPVariable_Wrap(out);
  });
}

// The cache: a tuple (k, k_scale, v, v_scale).
struct Cache {
  const Tensor *k, *ks, *v, *vs;
  sparq24_kvcache c;
};
Cache cache_of(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) type_error("cache must be a KVCache (k, k_scale, v, v_scale)");
  Cache x{&tensor(PyTuple_GET_ITEM(o, 0), "cache.k"), &tensor(PyTuple_GET_ITEM(o, 1), "cache.k_scale"),
          &tensor(PyTuple_GET_ITEM(o, 2), "cache.v"), &tensor(PyTuple_GET_ITEM(o, 3), "cache.v_scale"), {}};
  const Tensor &k = *x.k, &v = *x.v;
  if (k.dim() != 4 || v.dim() != 4)
    value_error("cache codes must be [blocks, heads, tokens, dim] and [blocks, heads, dim, tokens]");
  const int64_t blocks = k.size(0), heads = k.size(1), tokens = k.size(2), dim = k.size(3);
  if (v.size(0) != blocks || v.size(1) != heads || v.size(2) != dim || v.size(3) != tokens ||
      k.scalar_type() != v.scalar_type())
    value_error("cache codes " + shape_of(k) + " and " + shape_of(v) + " do not match");
  if (k.scalar_type() != ScalarType::Char && k.scalar_type() != ScalarType::Byte)
    type_error("cache codes are int8 or uint8 (e4m3), got " + shape_of(k));
  if (!k.is_contiguous() || !v.is_contiguous()) value_error("cache codes must be contiguous");
  x.c = {k.data_ptr(), vector<float>(*x.ks, blocks * heads, ScalarType::Float, "k_scale"),
         v.data_ptr(), vector<float>(*x.vs, blocks * heads, ScalarType::Float, "v_scale"),
         k.scalar_type() == ScalarType::Char ? SPARQ24_Q_INT : SPARQ24_Q_FP8_E4M3,
         blocks, heads, tokens, dim};
  return x;
}

// The sequences of token rows x: [total, heads, dim] with cu, or [seqs, n, heads, dim].
sparq24_kvseqs seqs_of(const Tensor& x, const Tensor& table, const Tensor& lens, const Tensor* cu) {
  if (table.dim() != 2 || table.scalar_type() != ScalarType::Int)
    value_error("block_table must be int32 [seqs, max blocks]");
  const int64_t seqs = table.size(0), width = table.size(1);
  if (width > 1 && table.stride(1) != 1) value_error("block_table must have contiguous rows");
  int64_t total;
  const int32_t* pcu = nullptr;
  if (cu) {
    if (x.dim() != 3) value_error("with cu_tokens token rows are [total, heads, dim], got " + shape_of(x));
    total = x.size(0);
    pcu = vector<int32_t>(*cu, seqs + 1, ScalarType::Int, "cu_tokens");
  } else {
    if (x.dim() != 4 || x.size(0) != seqs)
      value_error("without cu_tokens token rows are [seqs, n, heads, dim], got " + shape_of(x));
    total = seqs * x.size(1);
  }
  return {width ? (const int32_t*)table.data_ptr() : nullptr, width, table.stride(0),
          vector<int32_t>(lens, seqs, ScalarType::Int, "seq_lens"), pcu, seqs, total};
}

// Token rows: one batch entry per token.
sparq24_tensor rows_of(const Tensor& x) {
  const int code = dtype_code(x.scalar_type());
  int64_t total = x.size(0), step = x.stride(0);
  if (x.dim() == 4) {
    const int64_t a = x.size(0), n = x.size(1);
    if (a > 1 && n > 1 && x.stride(0) != n * x.stride(1))
      value_error("the sequences of token rows must be evenly spaced (or contiguous)");
    total = a * n;
    step = n > 1 ? x.stride(1) : x.stride(0);
  }
  if (x.size(-1) > 1 && x.stride(-1) != 1) value_error("token rows must be contiguous along dim");
  return {x.data_ptr(), code, total, x.size(-2), x.size(-1), step, x.stride(-2), 1};
}

// kv_append(cache, k, v, block_table, seq_lens, cu_tokens)
PyObject* py_kv_append(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    arguments(argc, 6);
    const Cache c = cache_of(a[0]);
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &table = tensor(a[3], "block_table");
    const Tensor &lens = tensor(a[4], "seq_lens"), *cu = optional(a[5], "cu_tokens");
    if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
      value_error("k " + shape_of(k) + " and v " + shape_of(v) + " do not match");
    const sparq24_kvseqs q = seqs_of(k, table, lens, cu);
    const sparq24_tensor kr = rows_of(k), vr = rows_of(v);
    const int dev = device_of({&k, &v, &table, &lens, cu, c.k, c.ks, c.v, c.vs});
    const int st = on_device(dev, [&](hipStream_t s) { return c_kv_append(&c.c, &q, &kr, &vr, s); });
    if (st) return failed("sparq24_kv_append", st);
    Py_RETURN_NONE;
  });
}

// kv_attention(q, cache, block_table, seq_lens, cu_tokens, scale or None, causal, window, return_lse, out, lse,
//              workspace) -> out or (out, lse)
PyObject* py_kv_attention(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    arguments(argc, 12);
    const Tensor& q = tensor(a[0], "q");
    const Cache c = cache_of(a[1]);
    const Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
    const Tensor *cu = optional(a[4], "cu_tokens"), *gout = optional(a[9], "out"), *glse = optional(a[10], "lse");
    const Tensor* work = optional(a[11], "workspace");
    const sparq24_kvseqs s = seqs_of(q, table, lens, cu);
    const sparq24_tensor x = rows_of(q);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)q.size(-1)) : PyFloat_AsDouble(a[5]);
    const int causal = PyObject_IsTrue(a[6]);
    const long long window = PyLong_AsLongLong(a[7]);
    const int want_lse = PyObject_IsTrue(a[8]);
    if (PyErr_Occurred()) return nullptr;
    if (gout && (gout->sizes() != q.sizes() || gout->scalar_type() != q.scalar_type() || !gout->is_contiguous()))
      value_error("out must be contiguous, of q's shape and type");
    const auto rows = q.sizes().slice(0, q.dim() - 1);
    if (glse && (glse->sizes() != rows || glse->scalar_type() != ScalarType::Float || !glse->is_contiguous()))
      value_error("lse must be contiguous fp32 of q's shape without dim");
    if (work && !work->is_contiguous()) value_error("workspace must be contiguous");
    const int dev = device_of({&q, &table, &lens, cu, gout, glse, work, c.k, c.ks, c.v, c.vs});
    const Tensor out = gout ? *gout : at::empty(q.sizes(), q.options());
    const Tensor lse = glse ? *glse : (want_lse ? at::empty(rows, q.options().dtype(ScalarType::Float)) : Tensor());
    float* plse = lse.defined() ? (float*)lse.data_ptr() : nullptr;
    Tensor ws = work ? *work : Tensor();
    const int st = on_device(dev, [&](hipStream_t stream) -> int {
      auto call = [&](void* w, size_t* n) {
        return c_kv_attention(&c.c, &s, &x, (float)scale, causal, window, out.data_ptr(), plse, w, n, stream);
      };
      size_t n = work ? work->nbytes() : 0;
      if (!work) {
        const int e = call(nullptr, &n);
        if (e) return e;
        if (n) ws = at::empty({(int64_t)n}, q.options().dtype(ScalarType::Byte));
      }
      // without memory no size either: that would be the size query
      return n ? call(ws.data_ptr(), &n) : call(nullptr, nullptr);
    });
    if (st) return failed("sparq24_kv_attention", st);
    if (!want_lse) return THPVariable_Wrap(out);
    PyObject* pair = PyTuple_New(2);
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
    return pair;
  });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)())py_bind, METH_FASTCALL, nullptr},
    {"int8_gemm", (PyCFunction)(void (*)())py_int8_gemm, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)())py_kv_append, METH_FASTCALL, nullptr},
    {"kv_attention", (PyCFunction)(void (*)())py_kv_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
