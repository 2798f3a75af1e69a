// The Python side of the operators around the projection: tensors in, their
// checks, outputs allocated by PyTorch, one call of the C ABI on the current
// (or the given) stream.  Compiled, because a single-token call takes the GPU a
// few microseconds and the checks alone took longer than that in Python.
//
// Each function takes its arguments by position, None where one is left out,
// and returns the outputs or, where the library refuses, its status code;
// operators.py gives them names, defaults and exceptions.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "splitk.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A refusal, as the Python exception it becomes.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

const char* name_of(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "bfloat16";
    case ScalarType::Half: return "float16";
    case ScalarType::Float: return "float32";
    case ScalarType::Char: return "int8";
    case ScalarType::Long: return "int64";
    default: return c10::toString(t);
  }
}

int code_of(ScalarType t) {
  return t == ScalarType::Float ? SPLITK_DTYPE_F32 : t == ScalarType::Half ? SPLITK_DTYPE_F16 : SPLITK_DTYPE_BF16;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

// Argument `o` as a tensor; null where it is None.
const Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& required(PyObject* o, const char* name) {
  const Tensor* t = optional(o, name);
  if (t == nullptr) type_error(std::string(name) + " must be a tensor");
  return *t;
}

void want_type(const Tensor& t, const char* name, std::initializer_list<ScalarType> allowed) {
  std::string names;
  for (ScalarType a : allowed) {
    if (t.scalar_type() == a) return;
    names += (names.empty() ? "" : " or ") + std::string(name_of(a));
  }
  type_error(std::string(name) + " must be " + names + ", not " + name_of(t.scalar_type()));
}

// Operand t (if there) is on `device`, which is a GPU.
void want_device(const Tensor* t, const char* name, const at::Device& device) {
  if (t != nullptr && t->device() != device) {
    value_error(std::string(name) + " must be on " + device.str() + ", the operands' device");
  }
}
void want_gpu(const at::Device& device) {
  if (!device.is_cuda()) value_error("operands must be CUDA tensors");
}

// An operand or output that is there: contiguous, of this shape and type.
void want_whole(const Tensor& t, const char* name, at::IntArrayRef shape, ScalarType type, const at::Device& device) {
  if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous()) {
    value_error(std::string(name) + " must be a contiguous " + name_of(type) + " tensor of shape " + shape_text(shape));
  }
  want_device(&t, name, device);
}

// An output: the one given, or a new one.
struct Output {
  const Tensor* given = nullptr;
  Tensor made;
  void check(const char* name, at::IntArrayRef shape, ScalarType type, const at::Device& device) const {
    if (given != nullptr) want_whole(*given, name, shape, type, device);
  }
  void* data(at::IntArrayRef shape, ScalarType type, const at::Device& device) {
    if (given != nullptr) return given->data_ptr();
    made = Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
    return made.data_ptr();
  }
  PyObject* wrap() const { return THPVariable_Wrap(given != nullptr ? *given : made); }
};

// A tensor read as rows along its last dimension: [M, D] with contiguous rows any
// distance apart, or a contiguous [L, M, D].
struct Rows {
  int64_t rows, width, stride;
  Rows(const Tensor& t, const char* name) {
    const int64_t dims = t.dim();
    if (dims == 3 && t.is_contiguous()) {
      rows = t.size(0) * t.size(1);
      width = stride = t.size(2);
      return;
    }
    if (dims == 2 && (t.is_contiguous() || t.stride(1) == 1 || t.size(1) == 1)) {
      rows = t.size(0);
      width = t.size(1);
      stride = rows > 1 && !t.is_contiguous() ? t.stride(0) : width;
      return;
    }
    value_error(std::string(name) + " is [M, D] with contiguous rows, or a contiguous [L, M, D]");
  }
};

int as_int(int64_t v) { return v > INT32_MAX ? -1 : (int)v; }       // a size the library refuses

// The stream argument, or the device's current stream.
struct Stream {
  c10::cuda::CUDAStream stream;
  bool given;
  splitk_stream_t handle() const { return reinterpret_cast<splitk_stream_t>(stream.stream()); }
};
Stream stream_of(PyObject* o, const at::Device& device) {
  if (o == Py_None) return {c10::cuda::getCurrentCUDAStream(device.index()), false};
  PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
  if (handle == nullptr) throw python_error();
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (p == nullptr && PyErr_Occurred()) throw python_error();
  return {c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), device.index()), true};
}

// What a call is enqueued under: Python may run other threads while memory is
// found and the call enqueued; the operands' device is the current one, and a stream
// given is its current stream, so that outputs made here are of that stream's
// memory: a block freed on another stream may still be in use there, and this
// one's, freed in turn, must not go to another while this one writes it.
struct Enqueue {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  c10::cuda::CUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard current;
  Enqueue(const at::Device& device, const Stream& s) : guard(device) {
    if (s.given) current.reset_stream(s.stream);
  }
};

PyObject* none() { return Py_NewRef(Py_None); }

// f(args), with what it throws as a Python exception.
template <class F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, q, scale, residual_out, stream)
PyObject* rmsnorm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rmsnorm_i8", n, 8, [&]() -> PyObject* {
    const Tensor &x = required(a[0], "x"), &weight = required(a[1], "weight");
    const Tensor* residual = optional(a[2], "residual");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    Output q{optional(a[4], "q"), {}}, scale{optional(a[5], "scale"), {}}, out{optional(a[6], "residual_out"), {}};
    const Rows r(x, "x");
    want_type(x, "x", {ScalarType::BFloat16});
    want_type(weight, "weight", {ScalarType::BFloat16, ScalarType::Float});
    if (weight.sizes() != at::IntArrayRef{r.width} || !weight.is_contiguous()) {
      value_error("weight must be a contiguous tensor of shape " + shape_text({r.width}));
    }
    const at::Device device = x.device();
    want_device(&weight, "weight", device);
    want_device(residual, "residual", device);
    want_gpu(device);
    const at::IntArrayRef shape = x.sizes(), rows = shape.slice(0, shape.size() - 1);
    ScalarType r_type = ScalarType::BFloat16;
    if (residual != nullptr) {
      want_type(*residual, "residual", {ScalarType::BFloat16, ScalarType::Float});
      r_type = residual->scalar_type();
      want_whole(*residual, "residual", shape, r_type, device);
      out.check("residual_out", shape, r_type, device);
    } else if (out.given != nullptr) {
      value_error("residual_out needs a residual");
    }
    q.check("q", shape, ScalarType::Char, device);
    scale.check("scale", rows, ScalarType::Float, device);
    const Stream stream = stream_of(a[7], device);
    int rc;
    {
      const Enqueue enqueue(device, stream);
      rc = splitk_rmsnorm_i8(x.data_ptr(), r.stride, residual ? residual->data_ptr() : nullptr,
                             residual ? out.data(shape, r_type, device) : nullptr, code_of(r_type), weight.data_ptr(),
                             code_of(weight.scalar_type()), (float)eps, q.data(shape, ScalarType::Char, device),
                             static_cast<float*>(scale.data(rows, ScalarType::Float, device)), as_int(r.rows),
                             as_int(r.width), stream.handle());
    }
    if (rc != SPLITK_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("NNN", q.wrap(), scale.wrap(), residual ? out.wrap() : none());
  });
}

// (x, q, scale, stream)
PyObject* quantize_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("quantize_i8", n, 4, [&]() -> PyObject* {
    const Tensor& x = required(a[0], "x");
    Output q{optional(a[1], "q"), {}}, scale{optional(a[2], "scale"), {}};
    const Rows r(x, "x");
    want_type(x, "x", {ScalarType::BFloat16});
    const at::Device device = x.device();
    want_gpu(device);
    const at::IntArrayRef shape = x.sizes(), rows = shape.slice(0, shape.size() - 1);
    q.check("q", shape, ScalarType::Char, device);
    scale.check("scale", rows, ScalarType::Float, device);
    const Stream stream = stream_of(a[3], device);
    int rc;
    {
      const Enqueue enqueue(device, stream);
      rc = splitk_quantize_i8(x.data_ptr(), r.stride, q.data(shape, ScalarType::Char, device),
                              static_cast<float*>(scale.data(rows, ScalarType::Float, device)), as_int(r.rows),
                              as_int(r.width), stream.handle());
    }
    if (rc != SPLITK_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("NN", q.wrap(), scale.wrap());
  });
}

// (a_q, a_scale, b_q, b_scale, c, bias, out_dtype, stream)
PyObject* gemm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gemm_i8", n, 8, [&]() -> PyObject* {
    const Tensor &a_q = required(a[0], "a_q"), &a_scale = required(a[1], "a_scale"), &b_q = required(a[2], "b_q"),
                 &b_scale = required(a[3], "b_scale");
    Output c{optional(a[4], "c"), {}};
    const Tensor* bias = optional(a[5], "bias");
    want_type(a_q, "a_q", {ScalarType::Char});
    want_type(b_q, "b_q", {ScalarType::Char});
    want_type(a_scale, "a_scale", {ScalarType::Float});
    want_type(b_scale, "b_scale", {ScalarType::Float});
    const int64_t dims = a_q.dim();
    if ((dims != 2 && dims != 3) || b_q.dim() != dims) {
      value_error("a_q is [L, N, K] or [N, K]; b_q is [L, M, K] or [M, K]");
    }
    const at::IntArrayRef as = a_q.sizes(), bs = b_q.sizes();
    const int64_t L = dims == 3 ? as[0] : 1, N = as[dims - 2], M = bs[dims - 2], K = as[dims - 1];
    const int64_t batched[3] = {L, M, N};
    const at::IntArrayRef outputs(batched + (3 - dims), dims);
    if (bs[dims - 1] != K || (dims == 3 && bs[0] != L) || a_scale.sizes() != as.slice(0, dims - 1) ||
        b_scale.sizes() != bs.slice(0, dims - 1)) {
      value_error("shape mismatch: a_q" + shape_text(as) + " a_scale" + shape_text(a_scale.sizes()) + " b_q" +
                  shape_text(bs) + " b_scale" + shape_text(b_scale.sizes()));
    }
    if (!a_q.is_contiguous() || !a_scale.is_contiguous() || !b_q.is_contiguous() || !b_scale.is_contiguous()) {
      value_error("operands must be contiguous");
    }
    const at::Device device = a_q.device();
    want_device(&a_scale, "a_scale", device);
    want_device(&b_q, "b_q", device);
    want_device(&b_scale, "b_scale", device);
    want_device(bias, "bias", device);
    want_gpu(device);
    if (bias != nullptr) want_whole(*bias, "bias", as.slice(0, dims - 1), ScalarType::BFloat16, device);
    ScalarType type = c.given != nullptr ? c.given->scalar_type() : ScalarType::BFloat16;
    if (a[6] != Py_None) {
      if (!THPDtype_Check(a[6])) type_error("out_dtype must be a torch.dtype");
      type = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
    }
    if (type != ScalarType::BFloat16 && type != ScalarType::Float) {
      type_error(std::string("c must be bfloat16 or float32, not ") + name_of(type));
    }
    c.check("c", outputs, type, device);
    const Stream stream = stream_of(a[7], device);
    int rc;
    {
      const Enqueue enqueue(device, stream);
      rc = splitk_gemm_i8(a_q.data_ptr(), a_scale.data_ptr<float>(), b_q.data_ptr(), b_scale.data_ptr<float>(),
                          bias ? bias->data_ptr() : nullptr, c.data(outputs, type, device), code_of(type), as_int(M),
                          as_int(N), as_int(K), as_int(L), stream.handle());
    }
    if (rc != SPLITK_OK) return PyLong_FromLong(rc);
    return c.wrap();
  });
}

// (logits, tokens, top_k, logprob, entropy, top_ids, top_logprobs, stream)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("logprobs", n, 8, [&]() -> PyObject* {
    const Tensor& logits = required(a[0], "logits");
    const Tensor* tokens = optional(a[1], "tokens");
    const Py_ssize_t k = PyNumber_AsSsize_t(a[2], PyExc_OverflowError);
    if (k == -1 && PyErr_Occurred()) throw python_error();
    Output logprob{optional(a[3], "logprob"), {}}, entropy{optional(a[4], "entropy"), {}},
        ids{optional(a[5], "top_ids"), {}}, tops{optional(a[6], "top_logprobs"), {}};
    const Rows r(logits, "logits");
    want_type(logits, "logits", {ScalarType::BFloat16, ScalarType::Half, ScalarType::Float});
    const at::Device device = logits.device();
    want_device(tokens, "tokens", device);
    want_gpu(device);
    const at::IntArrayRef rows = logits.sizes().slice(0, logits.dim() - 1);
    if (tokens != nullptr) {
      want_whole(*tokens, "tokens", rows, ScalarType::Long, device);
      logprob.check("logprob", rows, ScalarType::Float, device);
    } else if (logprob.given != nullptr) {
      value_error("logprob needs tokens");
    }
    entropy.check("entropy", rows, ScalarType::Float, device);
    // a count the library refuses is not allocated for
    const bool some = k > 0 && k <= r.width && k <= 1024;
    int64_t sized[3] = {rows[0], rows.size() > 1 ? rows[1] : (int64_t)k, (int64_t)k};
    const at::IntArrayRef wide(sized, rows.size() + 1);
    if (some) {
      ids.check("top_ids", wide, ScalarType::Long, device);
      tops.check("top_logprobs", wide, ScalarType::Float, device);
    } else if (k == 0 && (ids.given != nullptr || tops.given != nullptr)) {
      value_error("the alternatives' outputs need top_k > 0");
    }
    const Stream stream = stream_of(a[7], device);
    int rc = SPLITK_ERR_INVALID_ARGUMENT;
    if (k == 0 || some) {
      const Enqueue enqueue(device, stream);
      rc = splitk_logprobs(logits.data_ptr(), code_of(logits.scalar_type()), r.stride,
                           tokens ? reinterpret_cast<const long long*>(tokens->data_ptr<int64_t>()) : nullptr,
                           tokens ? static_cast<float*>(logprob.data(rows, ScalarType::Float, device)) : nullptr,
                           static_cast<float*>(entropy.data(rows, ScalarType::Float, device)), (int)k,
                           some ? static_cast<long long*>(ids.data(wide, ScalarType::Long, device)) : nullptr,
                           some ? static_cast<float*>(tops.data(wide, ScalarType::Float, device)) : nullptr,
                           as_int(r.rows), as_int(r.width), stream.handle());
    }
    if (rc != SPLITK_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("NNNN", tokens ? logprob.wrap() : none(), entropy.wrap(), some ? ids.wrap() : none(),
                         some ? tops.wrap() : none());
  });
}

#define FASTCALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FASTCALL(rmsnorm_i8), FASTCALL(quantize_i8), FASTCALL(gemm_i8), FASTCALL(logprobs),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators(void) { return PyModule_Create(&module); }
