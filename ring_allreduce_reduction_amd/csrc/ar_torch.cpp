// ar_torch.cpp -- Python calls of the operators around the AllReduce.
//
// The operators take up to nine lists of tensors, one tensor a rank; reading
// their addresses and checking them through Python attributes takes several
// times as long as the kernels of a small call (8 ranks, 48 tensors: 30 us).
// This module reads torch's tensors directly.  It checks what the C side
// cannot -- element types, shapes, strides, devices -- and passes plain
// pointers and sizes on; all work runs in libar.so, whose entry points
// binding.py hands over with bind().
#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <vector>

#include "ar.h"

namespace {

typedef arResult_t (*LayerNormFn)(const void* const*, const void* const*, const void* const*, void* const*,
                                  float* const*, float* const*, const size_t*, int, size_t, size_t, size_t, float,
                                  arDataType_t, arDataType_t, void*);
typedef arResult_t (*LayerNormBackwardFn)(const void* const*, const void* const*, const void* const*,
                                          const float* const*, const float* const*, void* const*, void* const*,
                                          void* const*, const size_t*, int, size_t, size_t, size_t, size_t,
                                          arDataType_t, arDataType_t, void*, size_t, void*);
typedef arResult_t (*WorkspaceFn)(const size_t*, int, size_t, size_t*);
typedef arResult_t (*ListCreateFn)(arTensorList_t*, int, const void* const*, void* const*, const size_t*,
                                   const arDataType_t*);
typedef arResult_t (*GradNormFn)(arTensorList_t, arNormKind_t, float, float*, void*, size_t, void*);
typedef arResult_t (*GradClipFn)(arTensorList_t, arNormKind_t, float, float, float, float*, void*, size_t, void*);

LayerNormFn gLayerNorm;
LayerNormBackwardFn gLayerNormBackward;
WorkspaceFn gWorkspace;
ListCreateFn gListCreate;
GradNormFn gGradNorm;
GradClipFn gGradClip;

// A Python error is set and the call ends.
struct PythonError {};

template <typename... A>
[[noreturn]] void fail(const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw PythonError();
}

const char* typeName(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
  }
}

bool floatType(at::ScalarType t) { return t == at::kFloat || t == at::kHalf || t == at::kBFloat16; }

arDataType_t codeOf(at::ScalarType t) { return t == at::kFloat ? arFloat32 : t == at::kHalf ? arFloat16 : arBfloat16; }

const at::Tensor& tensorOf(PyObject* o) {
  if (!THPVariable_Check(o)) fail("expected a tensor, got %.80s", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// Every tensor of a call lives on the current device: the kernels run there.
struct Devices {
  int current = -1;
  bool anyHost = false;
  int other = -1;
  void see(const at::Tensor& t) {
    if (!t.is_cuda()) {
      anyHost = true;
      return;
    }
    if (t.is_neg()) fail("a tensor is a lazy negation: call resolve_neg() first");
    const int d = t.get_device();
    if (current < 0 && hipGetDevice(&current) != hipSuccess) current = -1;
    if (d != current) other = d;
  }
  void check() const {
    if (anyHost) fail("operator tensors must be device tensors");
    if (other >= 0) fail("a tensor is on cuda:%d, the current device is cuda:%d", other, current);
  }
};

// A list or tuple of tensors, one a rank unless `most` says otherwise.
struct List {
  PyObject* fast = nullptr;
  int n = 0;
  explicit List(PyObject* o, Py_ssize_t most = AR_MAX_RANKS) {
    if (THPVariable_Check(o)) fail("expected a list of tensors, got one tensor");   // it would be read row by row
    fast = PySequence_Fast(o, "expected a list of tensors");
    if (fast == nullptr) throw PythonError();
    const Py_ssize_t size = PySequence_Fast_GET_SIZE(fast);
    if (size > most) {
      Py_CLEAR(fast);
      fail("at most %zd tensors, got %zd", most, size);
    }
    n = (int)size;
  }
  ~List() { Py_XDECREF(fast); }
  List(const List&) = delete;
  List& operator=(const List&) = delete;
  const at::Tensor& operator[](int i) const { return tensorOf(PySequence_Fast_GET_ITEM(fast, i)); }
};

struct Call {
  int n = 0;
  int64_t cols = 0;
  at::ScalarType type = at::kFloat, weights = at::kFloat;
  size_t rows[AR_MAX_RANKS];
  Devices devices;

  // Element types and width from the ranks' rows and their first weights.
  void start(const List& xs, PyObject* const* w, int nw) {
    n = xs.n;
    if (n < 1) fail("need at least one rank");
    const at::Tensor& x = xs[0];
    type = x.scalar_type();
    if (!floatType(type) || x.dim() < 1)
      fail("rows must be float32, float16 or bfloat16 tensors of at least one dimension");
    cols = x.size(-1);
    if (cols < 1) fail("rows must have at least one column");
    weights = type;
    for (int i = 0; i < nw; ++i)
      if (w[i] != Py_None) {
        const List l(w[i]);
        if (l.n < 1) continue;
        weights = l[0].scalar_type();
        break;
      }
    if (weights != type && weights != at::kFloat)
      fail("weights must be %s or float32, got %s", typeName(type), typeName(weights));
  }

  // Row buffers: (..., cols), contiguous or 2-D with unit column stride and a
  // row stride that all ranks share.  `first`: these set the ranks' rows.
  size_t rowBuffers(const char* what, const List& l, void** out, bool first) {
    if (l.n != n) fail("need %d %s buffers, got %d", n, what, l.n);
    int64_t stride = -1;
    for (int r = 0; r < n; ++r) {
      const at::Tensor& t = l[r];
      const int64_t dim = t.dim();
      if (dim < 1 || t.size(-1) != cols)
        fail("%s buffer %d has %lld columns, expected rows of %lld", what, r,
             (long long)(dim < 1 ? 0 : t.size(-1)), (long long)cols);
      if (t.scalar_type() != type)
        fail("%s buffer %d is %s, expected %s like the others", what, r, typeName(t.scalar_type()), typeName(type));
      const int64_t k = dim == 2 ? t.size(0) : t.numel() / cols;
      if (first) rows[r] = (size_t)k;
      else if ((size_t)k != rows[r])
        fail("%s buffer %d has %lld rows, expected %lld", what, r, (long long)k, (long long)rows[r]);
      int64_t s = cols;
      if (!t.is_contiguous()) {
        if (dim != 2 || (cols > 1 && t.stride(1) != 1) || (k > 1 && t.stride(0) < cols))
          fail("%s buffer %d must have contiguous rows", what, r);
        s = t.stride(0);
      }
      if (k > 1) {
        if (stride < 0) stride = s;
        else if (stride != s)
          fail("%s buffer %d has row stride %lld, the others %lld", what, r, (long long)s, (long long)stride);
      }
      devices.see(t);
      out[r] = t.data_ptr();
    }
    return (size_t)(stride < 0 ? cols : stride);
  }

  // One dense buffer a rank, of cols elements or (perRow) one element a row;
  // null pointers to none.
  void flatBuffers(const char* what, PyObject* o, at::ScalarType t, bool perRow, void** out) {
    const List l(o);
    if (l.n != n) fail("need %d %s buffers, got %d", n, what, l.n);
    for (int r = 0; r < n; ++r) {
      const at::Tensor& b = l[r];
      const int64_t size = perRow ? (int64_t)rows[r] : cols;
      if (b.scalar_type() != t) fail("%s buffer %d is %s, expected %s", what, r, typeName(b.scalar_type()), typeName(t));
      if (!b.is_contiguous() || b.numel() != size)
        fail("%s buffer %d must hold %lld contiguous elements", what, r, (long long)size);
      devices.see(b);
      out[r] = b.data_ptr();
    }
  }
};

// The workspace tensor's address; None gives null (the C side refuses it where
// one is needed).
void* workspaceOf(PyObject* o, size_t need, Devices* devices) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensorOf(o);
  if (!t.is_contiguous() || (size_t)t.nbytes() < need)
    fail("the workspace must be contiguous and hold %zu bytes", need);
  if ((uintptr_t)t.data_ptr() % 16) fail("the workspace must be 16-byte aligned");
  devices->see(t);
  return t.data_ptr();
}

// A torch stream, a raw handle, or None: torch's current stream.  A stream of
// another device than the tensors' would run the kernels there.
void* streamOf(PyObject* o, const Devices& devices) {
  if (o == Py_None) return (void*)c10::hip::getCurrentHIPStream().stream();
  if (PyLong_Check(o)) {
    void* p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw PythonError();
    return p;
  }
  PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
  if (handle == nullptr) throw PythonError();
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (PyErr_Occurred()) throw PythonError();
  PyObject* index = PyObject_GetAttrString(o, "device_index");   // torch's streams have one
  if (index == nullptr) {
    PyErr_Clear();
    return p;
  }
  const long d = PyLong_AsLong(index);
  Py_DECREF(index);
  if (PyErr_Occurred()) throw PythonError();
  if (devices.current >= 0 && d != devices.current)
    fail("the stream is on cuda:%ld, the current device is cuda:%d", d, devices.current);
  return p;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <typename F>
PyObject* result(F call) {
  arResult_t r;
  Py_BEGIN_ALLOW_THREADS
  r = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)r);
}

bool arguments(Py_ssize_t given, Py_ssize_t want) {
  if (given == want && gLayerNorm != nullptr) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or called before bind()");
  return false;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  gLayerNorm = (LayerNormFn)p[0];
  gLayerNormBackward = (LayerNormBackwardFn)p[1];
  gWorkspace = (WorkspaceFn)p[2];
  gListCreate = (ListCreateFn)p[3];
  gGradNorm = (GradNormFn)p[4];
  gGradClip = (GradClipFn)p[5];
  Py_RETURN_NONE;
}

// layer_norm(xs, ys, gammas, betas, means, rstds, eps, stream) -> result code
PyObject* layerNorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    Call c;
    const List xs(args[0]);
    c.start(xs, args + 2, 2);
    void *x[AR_MAX_RANKS], *y[AR_MAX_RANKS], *g[AR_MAX_RANKS], *b[AR_MAX_RANKS], *m[AR_MAX_RANKS], *s[AR_MAX_RANKS];
    const size_t xStride = c.rowBuffers("input", xs, x, true);
    const List ys(args[1]);
    const size_t yStride = c.rowBuffers("output", ys, y, false);
    if ((args[4] == Py_None) != (args[5] == Py_None)) fail("give both means and rstds or neither");
    if (args[2] != Py_None) c.flatBuffers("gamma", args[2], c.weights, false, g);
    if (args[3] != Py_None) c.flatBuffers("beta", args[3], c.weights, false, b);
    const bool stats = args[4] != Py_None;
    if (stats) {
      c.flatBuffers("mean", args[4], at::kFloat, true, m);
      c.flatBuffers("rstd", args[5], at::kFloat, true, s);
    }
    c.devices.check();
    const float eps = (float)PyFloat_AsDouble(args[6]);
    if (PyErr_Occurred()) return nullptr;
    void* stream = streamOf(args[7], c.devices);
    return result([&] {
      return gLayerNorm(x, args[2] != Py_None ? g : nullptr, args[3] != Py_None ? b : nullptr, y,
                        stats ? (float**)m : nullptr, stats ? (float**)s : nullptr, c.rows, c.n, (size_t)c.cols,
                        xStride, yStride, eps, codeOf(c.type), codeOf(c.weights), stream);
    });
  });
}

// layer_norm_backward(dys, xs, means, rstds, gammas, dxs, dgammas, dbetas, workspace, stream) -> result code, or
// the bytes of workspace it needs as a negative number where workspace is None and it needs one
PyObject* layerNormBackward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    Call c;
    const List xs(args[1]);
    PyObject* const weights[3] = {args[4], args[6], args[7]};
    c.start(xs, weights, 3);
    void *x[AR_MAX_RANKS], *dy[AR_MAX_RANKS], *dx[AR_MAX_RANKS], *m[AR_MAX_RANKS], *s[AR_MAX_RANKS], *g[AR_MAX_RANKS],
        *dg[AR_MAX_RANKS], *db[AR_MAX_RANKS];
    const size_t xStride = c.rowBuffers("input", xs, x, true);
    const List dys(args[0]);
    const size_t dyStride = c.rowBuffers("output gradient", dys, dy, false);
    size_t dxStride = (size_t)c.cols;
    const bool hasDx = args[5] != Py_None;
    if (hasDx) {
      const List dxs(args[5]);
      dxStride = c.rowBuffers("input gradient", dxs, dx, false);
    }
    c.flatBuffers("mean", args[2], at::kFloat, true, m);
    c.flatBuffers("rstd", args[3], at::kFloat, true, s);
    if (args[4] != Py_None) c.flatBuffers("gamma", args[4], c.weights, false, g);
    const bool hasDg = args[6] != Py_None, hasDb = args[7] != Py_None;
    if (hasDg) c.flatBuffers("gamma gradient", args[6], c.weights, false, dg);
    if (hasDb) c.flatBuffers("beta gradient", args[7], c.weights, false, db);
    size_t need = 0;
    void* workspace = nullptr;
    if (hasDg || hasDb) {
      const arResult_t r = gWorkspace(c.rows, c.n, (size_t)c.cols, &need);
      if (r != arSuccess) return PyLong_FromLong((long)r);
      workspace = workspaceOf(args[8], need, &c.devices);
    }
    c.devices.check();
    if (need > 0 && workspace == nullptr) return PyLong_FromLongLong(-(long long)need);
    void* stream = streamOf(args[9], c.devices);
    return result([&] {
      return gLayerNormBackward(dy, x, args[4] != Py_None ? g : nullptr, (float**)m, (float**)s, hasDx ? dx : nullptr,
                                hasDg ? dg : nullptr, hasDb ? db : nullptr, c.rows, c.n, (size_t)c.cols, dyStride,
                                xStride, dxStride, codeOf(c.type), codeOf(c.weights), workspace, need, stream);
    });
  });
}

// tensor_list(srcs, dsts or None) -> (result code, list address)
PyObject* tensorList(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 2)) return nullptr;
  return guarded([&]() -> PyObject* {
    constexpr Py_ssize_t kMost = 1 << 20;
    const List srcs(args[0], kMost);
    const bool outputs = args[1] != Py_None;
    std::vector<const void*> src((size_t)srcs.n);
    std::vector<void*> dst(outputs ? (size_t)srcs.n + 1 : 0);   // never empty: null means no outputs
    std::vector<size_t> counts((size_t)srcs.n);
    std::vector<arDataType_t> types((size_t)srcs.n);
    Devices devices;
    for (int i = 0; i < srcs.n; ++i) {
      const at::Tensor& t = srcs[i];
      if (!floatType(t.scalar_type())) fail("tensor %d is %s", i, typeName(t.scalar_type()));
      if (!t.is_contiguous())
        fail("tensor %d must hold %lld contiguous elements of %s", i, (long long)t.numel(), typeName(t.scalar_type()));
      devices.see(t);
      src[(size_t)i] = t.data_ptr();
      counts[(size_t)i] = (size_t)t.numel();
      types[(size_t)i] = codeOf(t.scalar_type());
    }
    if (outputs) {
      const List dsts(args[1], kMost);
      if (dsts.n != srcs.n) fail("need %d outputs, got %d", srcs.n, dsts.n);
      for (int i = 0; i < srcs.n; ++i) {
        const at::Tensor &t = srcs[i], &o = dsts[i];
        if (!o.is_contiguous() || o.scalar_type() != t.scalar_type() || o.numel() != t.numel())
          fail("output %d must hold %lld contiguous elements of %s", i, (long long)t.numel(),
               typeName(t.scalar_type()));
        devices.see(o);
        dst[(size_t)i] = o.data_ptr();
      }
    }
    devices.check();
    arTensorList_t list = nullptr;
    const arResult_t r = gListCreate(&list, srcs.n, src.data(), outputs ? dst.data() : nullptr, counts.data(),
                                     types.data());
    PyObject* address = PyLong_FromVoidPtr(list);
    if (address == nullptr) return nullptr;
    return Py_BuildValue("(iN)", (int)r, address);
  });
}

// grad_norm(list address, its workspace bytes, kind, scale, maxNorm or None, eps, norm, workspace, stream) ->
// result code
PyObject* gradNorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    arTensorList_t list = (arTensorList_t)PyLong_AsVoidPtr(args[0]);
    const size_t need = PyLong_AsSize_t(args[1]);
    const arNormKind_t kind = (arNormKind_t)PyLong_AsLong(args[2]);
    const float scale = (float)PyFloat_AsDouble(args[3]);
    const bool clip = args[4] != Py_None;
    const float maxNorm = clip ? (float)PyFloat_AsDouble(args[4]) : 0.0f;
    const float eps = (float)PyFloat_AsDouble(args[5]);
    if (PyErr_Occurred()) return nullptr;
    Devices devices;
    float* norm = nullptr;
    if (args[6] != Py_None) {
      const at::Tensor& t = tensorOf(args[6]);
      if (t.scalar_type() != at::kFloat || t.numel() != 1) fail("norm must be a float32 tensor of one element");
      devices.see(t);
      norm = (float*)t.data_ptr();
    }
    void* workspace = workspaceOf(args[7], need, &devices);
    devices.check();
    void* stream = streamOf(args[8], devices);
    return result([&] {
      return clip ? gGradClip(list, kind, scale, maxNorm, eps, norm, workspace, need, stream)
                  : gGradNorm(list, kind, scale, norm, workspace, need, stream);
    });
  });
}

#define FAST(f) ((PyCFunction)(void (*)(void))(f))
PyMethodDef kMethods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                          {"layer_norm", FAST(layerNorm), METH_FASTCALL, nullptr},
                          {"layer_norm_backward", FAST(layerNormBackward), METH_FASTCALL, nullptr},
                          {"tensor_list", FAST(tensorList), METH_FASTCALL, nullptr},
                          {"grad_norm", FAST(gradNorm), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ar_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the Python and torch whose headers this was compiled with; the
// binding uses the module with no other.
PyMODINIT_FUNC PyInit__ar_torch(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", AR_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
