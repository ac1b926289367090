// Python binding of the hot entry points for torch tensors.
//
// A call of the C ABI takes up to eleven tensor descriptors; filling them from
// Python costs about 0.6 us each, more than the small operators' kernels take.
// Here they are filled from the tensors themselves. One template wraps any entry
// point from its signature: a `const pa_tensor*` takes a torch.Tensor or None,
// int32_t and float take numbers, and the last argument, the stream, takes a
// handle or None for the current stream of the current device. Each wrapper
// returns the pa_status.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <utility>

#include "pa.h"

namespace {

bool element_type(at::ScalarType t, int32_t* out) {
  switch (t) {
    case at::kHalf: *out = PA_F16; return true;
    case at::kBFloat16: *out = PA_BF16; return true;
    case at::kByte:
    case at::kFloat8_e4m3fn: *out = PA_FP8_E4M3; return true;
    case at::kInt: *out = PA_I32; return true;
    case at::kLong: *out = PA_I64; return true;
    case at::kFloat: *out = PA_F32; return true;
    default: return false;
  }
}

// One converted argument. Each returns false with a Python exception set.
template <typename T>
struct Arg;

template <>
struct Arg<const pa_tensor*> {
  pa_tensor desc;
  const pa_tensor* value = nullptr;
  bool from(PyObject* o) {
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!element_type(t.scalar_type(), &desc.dtype)) {
      PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
      return false;
    }
    if (t.dim() > PA_MAX_DIMS) {
      PyErr_SetString(PyExc_ValueError, "too many dims");
      return false;
    }
    desc.ndim = static_cast<int32_t>(t.dim());
    for (int i = 0; i < PA_MAX_DIMS; ++i) {
      desc.shape[i] = i < desc.ndim ? t.size(i) : 0;
      desc.strides[i] = i < desc.ndim ? t.stride(i) : 0;
    }
    desc.data = t.data_ptr();
    value = &desc;
    return true;
  }
};

template <>
struct Arg<int32_t> {
  int32_t value = 0;
  bool from(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
      PyErr_SetString(PyExc_OverflowError, "integer argument beyond 32 bits");
      return false;
    }
    value = static_cast<int32_t>(v);
    return true;
  }
};

template <>
struct Arg<float> {
  float value = 0.f;
  bool from(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    value = static_cast<float>(v);
    return true;
  }
};

template <>
struct Arg<pa_stream> {
  pa_stream value = nullptr;
  bool from(PyObject* o) {
    if (o == Py_None) {
      value = c10::cuda::getCurrentCUDAStream().stream();
      return true;
    }
    value = PyLong_AsVoidPtr(o);
    return !(value == nullptr && PyErr_Occurred());
  }
};

template <auto Fn, typename Sig = decltype(Fn)>
struct Wrap;

template <auto Fn, typename... A>
struct Wrap<Fn, pa_status (*)(A...)> {
  template <size_t... I>
  static PyObject* run(PyObject* const* args, std::index_sequence<I...>) {
    std::tuple<Arg<A>...> conv;
    if (!(std::get<I>(conv).from(args[I]) && ...)) return nullptr;
    pa_status s;
    Py_BEGIN_ALLOW_THREADS
    s = Fn(std::get<I>(conv).value...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
  }
  static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
      PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd",
                   static_cast<Py_ssize_t>(sizeof...(A)), n);
      return nullptr;
    }
    try {
      return run(args, std::index_sequence_for<A...>{});
    } catch (const std::exception& e) {  // from torch (no CUDA device, for one)
      PyErr_SetString(PyExc_RuntimeError, e.what());
      return nullptr;
    }
  }
};

#define PA_WRAP(NAME) \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Wrap<&NAME>::call)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {PA_WRAP(pa_reshape_and_cache),
                          PA_WRAP(pa_norm_rope_and_cache),
                          PA_WRAP(pa_pool_extend),
                          PA_WRAP(pa_pool_release),
                          PA_WRAP(pa_decode),
                          PA_WRAP(pa_decode_noalloc),
                          PA_WRAP(pa_decode_shared),
                          PA_WRAP(pa_prefill_chunk),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pa_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch(void) { return PyModule_Create(&kModule); }
