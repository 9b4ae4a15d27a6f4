// What the parts of the extension module _seq_native share: the checks of tensors, outputs, workspaces and streams of one
// call, and the marshalling of arguments.
#pragma once

#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/ttt.h"

// lm_native.cpp's part of the module: its methods, ended by an empty one, and the lookup of its entry points.
extern PyMethodDef lm_methods[];
bool lm_bind(void* lib);

namespace {

using at::Tensor;

[[maybe_unused]] std::string text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

[[maybe_unused]] const Tensor& tensor_of(const char* name, PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a CUDA (HIP) tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA (HIP) tensor");
  return t;
}
[[maybe_unused]] const Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor_of(name, o); }

// Other Python threads run while this one allocates or waits for a place in a stream's queue.
struct NoGil {
  PyThreadState* const state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

template <class F, class... A>
ttt_status enqueue(F* f, A... a) {
  const NoGil free;
  return f(a...);
}

// A tensor of the caller's that a call has written counts as changed: autograd refuses a gradient that needs its old
// values. (Tensors made in inference mode have no count.)
[[maybe_unused]] void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An output: the caller's tensor or a new one.
struct Out {
  Tensor t;
  PyObject* given = nullptr;
  void* p = nullptr;
  PyObject* object() const {  // a new reference, of an output that has been written
    if (!p) Py_RETURN_NONE;
    if (given) return written(THPVariable_Unpack(given)), Py_INCREF(given), given;
    return THPVariable_Wrap(t);
  }
};

struct Rows {
  const void* p = nullptr;
  long long stride = 0;
};

// The device, dtype and stream of one call, and the checks of its tensors against them.
class Call {
 public:
  Call(const char* name, const Tensor& x) : device_(x.device()), io_(x.scalar_type()), guard_(x.device()) {
    TORCH_CHECK_TYPE(io_ == at::kBFloat16 || io_ == at::kFloat, "unsupported I/O dtype ", io_, " of ", name);
    dt = io_ == at::kBFloat16 ? TTT_BF16 : TTT_F32;
    stream = c10::hip::getCurrentHIPStream(device_.index()).stream();
  }

  void* need(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype) const {
    same(name, t, shape, dtype);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.data_ptr();
  }
  void* io(const char* name, const Tensor& t, at::IntArrayRef shape) const { return need(name, t, shape, io_); }
  const float* f32(const char* name, const Tensor& t, at::IntArrayRef shape) const {
    return static_cast<const float*>(need(name, t, shape, at::kFloat));
  }
  // The same of tensors that may be left out.
  void* io(const char* name, const Tensor* t, at::IntArrayRef shape) const { return t ? io(name, *t, shape) : nullptr; }
  const float* f32(const char* name, const Tensor* t, at::IntArrayRef shape) const {
    return t ? f32(name, *t, shape) : nullptr;
  }
  const int* lengths(const Tensor* t, int64_t B) const {
    return t ? static_cast<const int*>(need("lengths", *t, {B}, at::kInt)) : nullptr;
  }

  // An activation whose last dims (`width` elements) are contiguous and whose leading dims are one run of
  // evenly spaced rows.
  Rows rows(const char* name, const Tensor& t, at::IntArrayRef shape, int64_t width) const {
    same(name, t, shape, io_);
    if (t.is_contiguous()) return {t.data_ptr(), width};
    const auto sizes = t.sizes(), strides = t.strides();
    int d = (int)sizes.size();
    for (int64_t inner = 1; inner < width;) {  // the dims that make up a row
      --d;
      TORCH_CHECK_VALUE(sizes[d] == 1 || strides[d] == inner, "the last ", width, " elements of each row of ", name,
                        " must be contiguous");
      inner *= sizes[d];
    }
    int64_t step = -1, span = 0;
    for (int i = d - 1; i >= 0; --i) {
      if (sizes[i] == 1) continue;
      if (step < 0) step = strides[i];
      else TORCH_CHECK_VALUE(strides[i] == span, "the rows of ", name, " must be evenly spaced over its leading dims");
      span = strides[i] * sizes[i];
    }
    if (step < 0) step = width;
    TORCH_CHECK_VALUE(step >= width, "the rows of ", name, " overlap");
    return {t.data_ptr(), step};
  }

  // An output of `like`'s shape and dtype, or of these. (From the allocator directly, as the workspace is: through the
  // dispatcher it takes longer.)
  Out out(const char* name, PyObject* given, const Tensor& like) const {
    return out(name, given, like.sizes(), like.scalar_type());
  }
  Out out(const char* name, PyObject* given, at::IntArrayRef sizes, at::ScalarType dtype) const {
    Out o;
    if (given != Py_None) {
      const Tensor& t = tensor_of(name, given);
      o.p = need(name, t, sizes, dtype);
      o.given = given;
    } else {
      const NoGil free;
      o.t = at::detail::empty_cuda(sizes, dtype, device_, c10::nullopt);
      o.p = o.t.data_ptr();
    }
    return o;
  }
  // The gradient of an input, none where that is not there.
  Out grad(const char* name, PyObject* given, const Tensor* of) const {
    if (of) return out(name, given, *of);
    TORCH_CHECK_VALUE(given == Py_None, name, " is given without its input");
    return Out{};
  }

  // Pointer and bytes; `held` keeps a new one until the call is enqueued (its memory is given back in the order
  // of the stream).
  void* workspace(PyObject* given, size_t need, size_t& bytes, c10::DataPtr& held) const {
    bytes = 0;
    if (given != Py_None) {
      TORCH_CHECK_VALUE(THPVariable_Check(given) && THPVariable_Unpack(given).device() == device_ &&
                            THPVariable_Unpack(given).is_contiguous(),
                        "workspace must be a contiguous tensor on ", device_);
      const Tensor& t = THPVariable_Unpack(given);
      bytes = (size_t)t.numel() * t.element_size();
      return t.data_ptr();
    }
    if (need == 0) return nullptr;
    const NoGil free;
    held = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(need);
    bytes = need;
    return held.get();
  }

  ttt_dtype dt;
  hipStream_t stream;

 private:
  void same(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype) const {
    TORCH_CHECK_VALUE(t.device() == device_, name, " is on ", t.device(), ", not ", device_);
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, " must have dtype ", dtype, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(!t.is_neg(), name, " is a negated view: resolve_neg() it first");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", text(shape), ", not ", text(t.sizes()));
  }
  const at::Device device_;
  const at::ScalarType io_;
  const c10::DeviceGuard guard_;
  const at::AutoDispatchBelowADInplaceOrView below_;  // (outputs are new memory: autograd has no part in them)
};

// Sizes go to the C ABI as int: one that does not fit is refused here.
[[maybe_unused]] int as_int(const char* name, int64_t v) {
  TORCH_CHECK_VALUE(v >= 0 && v <= 0x7fffffff, name, " is too large: ", v);
  return (int)v;
}
[[maybe_unused]] bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}
[[maybe_unused]] double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
[[maybe_unused]] float number(PyObject* o) { return (float)real(o); }
[[maybe_unused]] PyObject* status(ttt_status st) { return PyLong_FromLong(st); }

template <size_t N>
PyObject* tuple_of(const Out (&outs)[N]) {
  PyObject* r = PyTuple_New(N);
  if (!r) throw python_error();
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, outs[i].object());
  return r;
}

// ---- norms over rows ---------------------------------------------------------------------------
struct Norm {
  int M, H, D;
};
// weight [D] norms x's rows, weight [H, D] each head's D of [..., H, D].
[[maybe_unused]] Norm norm_of(const Tensor& x, const Tensor& weight) {
  const auto ws = weight.sizes();
  const size_t nd = ws.size();
  TORCH_CHECK_VALUE(nd == 1 || nd == 2, "weight must be [D] or [H, D]");
  TORCH_CHECK_VALUE((size_t)x.dim() > nd && x.sizes().slice(x.dim() - nd) == ws, "x must be [...", nd == 2 ? ", H" : "",
                    ", D] for a weight of ", text(ws), ", not ", text(x.sizes()));
  const int64_t H = nd == 1 ? 1 : ws[0], D = ws[nd - 1], per = H * D;
  return {as_int("x", per ? x.numel() / per : 0), as_int("weight", H), as_int("weight", D)};
}

#define TTT_ARGS(n)                                                                        \
  if (count != n) {                                                                        \
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", n, count);           \
    return nullptr;                                                                        \
  }

#define TTT_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

// Looks an entry point of `api` up in a loaded libttt.so.
#define TTT_LOOKUP(name)                                                          \
  if (!(api.name = reinterpret_cast<decltype(api.name)>(dlsym(lib, #name)))) {    \
    PyErr_SetString(PyExc_RuntimeError, "libttt.so lacks " #name);                \
    return failed;                                                                \
  }

}  // namespace
