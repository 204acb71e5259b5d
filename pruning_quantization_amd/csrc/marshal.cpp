// Python marshalling of the calls that a serving step makes once per layer and
// token (rmsnorm_quantize, int8_gemm, mxfp4_gemm, kv_append, kv_attention): checks of the tensors, the C
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
decltype(&sparq24_mxfp4_gemm) c_mxfp4_gemm = nullptr;
decltype(&sparq24_rmsnorm_quantize) c_rmsnorm_quantize = nullptr;
decltype(&sparq24_kv_append_mxfp4) c_kv_append_mxfp4 = nullptr;
decltype(&sparq24_kv_attention_mxfp4) c_kv_attention_mxfp4 = nullptr;

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

// Scale bytes of rows of codes: their leading dims, or all rows in one, and then the groups.
uint8_t* scales(const Tensor& t, const Tensor& codes, int64_t rows, int64_t groups, const char* name) {
  const auto lead = codes.sizes().slice(0, codes.dim() - 1);
  const bool alike = t.dim() == codes.dim() && t.sizes().slice(0, t.dim() - 1) == lead;
  if (t.dim() < 1 || t.size(-1) != groups || !(alike || (t.dim() == 2 && t.size(0) == rows)))
    value_error(std::string(name) + " must be [..., K / 32] beside codes " + shape_of(codes) + ", got " + shape_of(t));
  return vector<uint8_t>(t, rows * groups, ScalarType::Byte, name);
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

// bind(addresses of sparq24_int8_gemm, _kv_append, _kv_attention, _mxfp4_gemm, _rmsnorm_quantize, _kv_append_mxfp4
// and _kv_attention_mxfp4, error class)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arguments(n, 8);
    c_int8_gemm = (decltype(c_int8_gemm))PyLong_AsVoidPtr(a[0]);
    c_kv_append = (decltype(c_kv_append))PyLong_AsVoidPtr(a[1]);
    c_kv_attention = (decltype(c_kv_attention))PyLong_AsVoidPtr(a[2]);
    c_mxfp4_gemm = (decltype(c_mxfp4_gemm))PyLong_AsVoidPtr(a[3]);
    c_rmsnorm_quantize = (decltype(c_rmsnorm_quantize))PyLong_AsVoidPtr(a[4]);
    c_kv_append_mxfp4 = (decltype(c_kv_append_mxfp4))PyLong_AsVoidPtr(a[5]);
    c_kv_attention_mxfp4 = (decltype(c_kv_attention_mxfp4))PyLong_AsVoidPtr(a[6]);
    if (PyErr_Occurred()) return nullptr;
    Py_XDECREF(call_error);
    call_error = Py_NewRef(a[7]);
    Py_RETURN_NONE;
  });
}

// A product of rows of codes, C = A B^T: what int8_gemm and mxfp4_gemm have in common.
// args: codes_a, scale_a, codes_b, scale_b, bias, dtype, out; width: the codes' dim.
struct Product {
  const Tensor &ca, &sa, &cb, &sb;
  const Tensor *bias, *given;
  int64_t m = 1, n, width, lda, ldb, ldc;
  ScalarType want;
  int code;
  float* pbias;
  std::vector<int64_t> shape;

  Product(PyObject* const* a, Py_ssize_t argc, ScalarType codes, const char* what)
      : ca(tensor((arguments(argc, 7), a[0]), "codes_a")), sa(tensor(a[1], "scale_a")), cb(tensor(a[2], "codes_b")),
        sb(tensor(a[3], "scale_b")), bias(optional(a[4], "bias")), given(optional(a[6], "out")) {
    if (ca.scalar_type() != codes || cb.scalar_type() != codes)
      type_error(std::string(what) + " codes expected, got " + shape_of(ca) + " and " + shape_of(cb));
    const int64_t rank = ca.dim();
    if (cb.dim() != 2 || rank < 1 || ca.size(-1) != cb.size(1))
      value_error("shapes " + shape_of(ca) + " and " + shape_of(cb) + " do not multiply");
    n = cb.size(0), width = cb.size(1);
    for (int64_t i = 0; i + 1 < rank; ++i) m *= ca.size(i);
    lda = rows(ca, width, "codes_a"), ldb = n > 1 ? cb.stride(0) : width;
    if (width > 1 && n && cb.stride(1) != 1) value_error("codes_b must be contiguous along K");
    if (!THPDtype_Check(a[5])) type_error("dtype must be a torch.dtype");
    want = given ? given->scalar_type() : ((THPDtype*)a[5])->scalar_type;
    code = dtype_code(want);
  }
  // Step between the m rows of t, whose leading dims have to be evenly spaced.
  int64_t rows(const Tensor& t, int64_t width, const char* name) const {
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
  }
  // The checks that follow those of the scales, and the output.
  template <class F>
  PyObject* run(const char* fn, F&& call) {
    pbias = bias ? vector<float>(*bias, n, ScalarType::Float, "bias") : nullptr;
    shape.assign(ca.sizes().begin(), ca.sizes().end());
    shape.back() = n;
    if (given && given->sizes() != at::IntArrayRef(shape)) value_error("out has shape " + shape_of(*given));
    ldc = given ? rows(*given, n, "out") : n;
    const int dev = device_of({&ca, &sa, &cb, &sb, bias, given});
    const Tensor out = given ? *given : at::empty(shape, ca.options().dtype(want));
    const int st = on_device(dev, [&](hipStream_t s) { return call(out.data_ptr(), s); });
    return st ? failed(fn, st) : THPVariable_Wrap(out);
  }
};

PyObject* py_int8_gemm(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Product p(a, argc, ScalarType::Char, "int8");
    float* psa = vector<float>(p.sa, p.m, ScalarType::Float, "scale_a");
    float* psb = vector<float>(p.sb, p.n, ScalarType::Float, "scale_b");
    return p.run("sparq24_int8_gemm", [&](void* out, hipStream_t s) {
      return c_int8_gemm((const int8_t*)p.ca.data_ptr(), p.lda, psa, p.m, (const int8_t*)p.cb.data_ptr(), p.ldb, psb,
                         p.n, p.width, p.pbias, p.code, out, p.ldc, nullptr, nullptr, s);
    });
  });
}

PyObject* py_mxfp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Product p(a, argc, ScalarType::Byte, "uint8 (two to a byte)");
    if (p.width % 16) value_error("rows of codes hold groups of 32 (16 bytes), got " + shape_of(p.ca));
    const int64_t groups = p.width / 16;
    uint8_t* psa = scales(p.sa, p.ca, p.m, groups, "scale_a");
    uint8_t* psb = scales(p.sb, p.cb, p.n, groups, "scale_b");
    return p.run("sparq24_mxfp4_gemm", [&](void* out, hipStream_t s) {
      return c_mxfp4_gemm((const uint8_t*)p.ca.data_ptr(), p.lda, psa, p.m, (const uint8_t*)p.cb.data_ptr(), p.ldb,
                          psb, p.n, 2 * p.width, p.pbias, p.code, out, p.ldc, nullptr, nullptr, s);
    });
  });
}

// Rows of t along its last dim: rows its second to last, batches the dims before, which have to be evenly spaced.
sparq24_tensor operand_of(const Tensor& t, const char* name) {
  const int64_t rank = t.dim();
  if (rank < 1) value_error(std::string(name) + " must have rows");
  if (t.size(-1) > 1 && t.stride(-1) != 1) value_error(std::string(name) + " must be contiguous along its last dim");
  int64_t batch = 1, step = 0;
  bool one = true;
  for (int64_t i = rank - 3; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (one) step = t.stride(i);
    else if (t.stride(i) != step * batch) value_error("the leading dims of " + std::string(name) + " must be evenly spaced");
    one = false;
    batch *= t.size(i);
  }
  return {t.data_ptr(), dtype_code(t.scalar_type()), batch, rank > 1 ? t.size(-2) : 1, t.size(-1),
          step, rank > 1 ? t.stride(-2) : t.size(-1), 1};
}

// rmsnorm_quantize(x, weight, fmt, bits, eps, residual, residual_out, codes, scales)
// -> (codes, scales) or (codes, scales, residual_out)
PyObject* py_rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    arguments(argc, 9);
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    sparq24_qspec q{(int32_t)PyLong_AsLong(a[2]), (int32_t)PyLong_AsLong(a[3]), nullptr};
    const double eps = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return nullptr;
    const Tensor *res = optional(a[5], "residual"), *gsum = optional(a[6], "residual_out");
    const Tensor *gcodes = optional(a[7], "codes"), *gscales = optional(a[8], "scales");
    const sparq24_tensor xt = operand_of(x, "x");
    const int64_t k = x.size(-1);
    if (w.dim() != 1 || w.numel() != k || !w.is_contiguous())
      value_error("weight must be contiguous with " + std::to_string(k) + " elements, got " + shape_of(w));
    const int wcode = dtype_code(w.scalar_type());
    if (gsum && !res) value_error("residual_out without a residual");
    sparq24_tensor rt{}, st{};
    if (res) {
      if (res->sizes() != x.sizes() || res->scalar_type() != x.scalar_type())
        value_error("residual " + shape_of(*res) + " is not of x's shape and type");
      if (gsum && (gsum->sizes() != x.sizes() || gsum->scalar_type() != x.scalar_type()))
        value_error("residual_out " + shape_of(*gsum) + " is not of x's shape and type");
      rt = operand_of(*res, "residual");
      if (gsum) st = operand_of(*gsum, "residual_out");
    }
    const bool mx = q.fmt == SPARQ24_Q_MXFP4;
    if (mx && k % 32) value_error("mxfp4 needs rows of 32 elements, got " + shape_of(x));
    std::vector<int64_t> cshape(x.sizes().begin(), x.sizes().end()), sshape(cshape);
    if (mx) cshape.back() = k / 2, sshape.back() = k / 32;
    else sshape.pop_back();
    const ScalarType ctype = q.fmt == SPARQ24_Q_INT ? ScalarType::Char : ScalarType::Byte;
    const ScalarType stype = mx ? ScalarType::Byte : ScalarType::Float;
    auto fits = [&](const Tensor* t, const std::vector<int64_t>& shape, ScalarType type, const char* name) {
      if (t && (t->sizes() != at::IntArrayRef(shape) || t->scalar_type() != type || !t->is_contiguous()))
        value_error(std::string(name) + " must be contiguous " + c10::toString(type) + " of the output's shape, got " +
                    shape_of(*t));
    };
    fits(gcodes, cshape, ctype, "codes");
    fits(gscales, sshape, stype, "scales");
    const int dev = device_of({&x, &w, res, gsum, gcodes, gscales});
    const Tensor codes = gcodes ? *gcodes : at::empty(cshape, x.options().dtype(ctype));
    const Tensor scales = gscales ? *gscales : at::empty(sshape, x.options().dtype(stype));
    Tensor sum;
    if (res) {
      sum = gsum ? *gsum : at::empty(x.sizes(), x.options());
      if (!gsum) st = operand_of(sum, "residual_out");
    }
    const int status = on_device(dev, [&](hipStream_t s) {
      return c_rmsnorm_quantize(&xt, res ? &rt : nullptr, w.data_ptr(), wcode, (float)eps, &q, codes.data_ptr(),
                                scales.data_ptr(), res ? &st : nullptr, s);
    });
    if (status) return failed("sparq24_rmsnorm_quantize", status);
    PyObject* t = PyTuple_New(res ? 3 : 2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(codes));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(scales));
    if (res) PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(sum));
    return t;
  });
}

// The cache: a tuple (k, k_scale, v, v_scale), of 8 bits or (uint8 scales) of 4.
struct Cache {
  const Tensor *k, *ks, *v, *vs;
  bool mx;
  sparq24_kvcache c;
  sparq24_kvcache_mxfp4 c4;
};
Cache cache_of(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) type_error("cache must be a KVCache (k, k_scale, v, v_scale)");
  Cache x{&tensor(PyTuple_GET_ITEM(o, 0), "cache.k"), &tensor(PyTuple_GET_ITEM(o, 1), "cache.k_scale"),
          &tensor(PyTuple_GET_ITEM(o, 2), "cache.v"), &tensor(PyTuple_GET_ITEM(o, 3), "cache.v_scale"), false, {}, {}};
  const Tensor &k = *x.k, &v = *x.v;
  x.mx = x.ks->scalar_type() == ScalarType::Byte;
  if (k.dim() != 4 || v.dim() != 4)
    value_error("cache codes must be [blocks, heads, tokens, dim] and [blocks, heads, dim, tokens] (4 bits: both "
                "[blocks, heads, tokens, dim / 2])");
  const int64_t blocks = k.size(0), heads = k.size(1), tokens = k.size(2), dim = k.size(3);
  if (v.size(0) != blocks || v.size(1) != heads || v.size(2) != (x.mx ? tokens : dim) ||
      v.size(3) != (x.mx ? dim : tokens) || k.scalar_type() != v.scalar_type())
    value_error("cache codes " + shape_of(k) + " and " + shape_of(v) + " do not match");
  if (x.mx ? k.scalar_type() != ScalarType::Byte
           : k.scalar_type() != ScalarType::Char && k.scalar_type() != ScalarType::Byte)
    type_error("cache codes are int8 or uint8 (e4m3; 4 bits, two to a byte), got " + shape_of(k));
  if (!k.is_contiguous() || !v.is_contiguous()) value_error("cache codes must be contiguous");
  if (x.mx) {
    const int64_t groups = dim / 16;
    for (const Tensor* t : {x.ks, x.vs})
      if (t->dim() != 4 || t->size(0) != blocks || t->size(1) != heads || t->size(2) != groups || t->size(3) != tokens)
        value_error("k_scale and v_scale of a 4-bit cache are [blocks, heads, dim / 32, tokens], got " + shape_of(*t));
    x.c4 = {(uint8_t*)k.data_ptr(), vector<uint8_t>(*x.ks, blocks * heads * groups * tokens, ScalarType::Byte, "k_scale"),
            (uint8_t*)v.data_ptr(), vector<uint8_t>(*x.vs, blocks * heads * groups * tokens, ScalarType::Byte, "v_scale"),
            blocks, heads, tokens, 2 * dim};
    return x;
  }
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
    const int st = on_device(dev, [&](hipStream_t s) {
      return c.mx ? c_kv_append_mxfp4(&c.c4, &q, &kr, &vr, s) : c_kv_append(&c.c, &q, &kr, &vr, s);
    });
    if (st) return failed(c.mx ? "sparq24_kv_append_mxfp4" : "sparq24_kv_append", st);
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
        if (c.mx)
          return c_kv_attention_mxfp4(&c.c4, &s, &x, (float)scale, causal, window, out.data_ptr(), plse, w, n, stream);
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
    if (st) return failed(c.mx ? "sparq24_kv_attention_mxfp4" : "sparq24_kv_attention", st);
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
    {"mxfp4_gemm", (PyCFunction)(void (*)())py_mxfp4_gemm, METH_FASTCALL, nullptr},
    {"rmsnorm_quantize", (PyCFunction)(void (*)())py_rmsnorm_quantize, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)())py_kv_append, METH_FASTCALL, nullptr},
    {"kv_attention", (PyCFunction)(void (*)())py_kv_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
