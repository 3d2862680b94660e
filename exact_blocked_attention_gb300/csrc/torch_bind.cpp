// Argument marshalling of the serving-step operators (rope, paged append,
// attention over pages) for torch tensors: descriptors straight from the
// tensor objects, outputs allocated, the current stream looked up, then one
// call into libblkattn's C ABI.  A decode step's kernels take a few
// microseconds; building nine descriptors in Python took longer than that.
//
// Holds no arithmetic and no state but the entry points' addresses.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "blkattn.h"

namespace {

decltype(&blkattn_rope) g_rope, g_rope_bwd;
decltype(&blkattn_paged_append) g_append;
decltype(&blkattn_fwd_paged) g_fwd;

// A descriptor of a tensor argument; None gives a NULL pointer.
class Desc {
 public:
  explicit Desc(PyObject* o) {
    if (o == Py_None) return;
    TORCH_CHECK_TYPE(THPVariable_Check(o), "blkattn: a tensor is wanted");
    init(THPVariable_Unpack(o));
  }
  explicit Desc(const at::Tensor& t) { init(t); }
  const blkattn_tensor* get() const { return given_ ? &d_ : nullptr; }
  bool given() const { return given_; }

 private:
  void init(const at::Tensor& t) {
    TORCH_CHECK_VALUE(t.layout() == at::kStrided, "blkattn: a strided tensor is wanted");
    TORCH_CHECK_VALUE(!t.is_neg() && !t.is_conj(), "blkattn: a negated view is not supported");
    switch (t.scalar_type()) {
      case at::kBFloat16: d_.dtype = BLKATTN_BF16; break;
      case at::kFloat: d_.dtype = BLKATTN_F32; break;
      case at::kInt: d_.dtype = BLKATTN_I32; break;
      case at::kLong: d_.dtype = BLKATTN_I64; break;
      default: TORCH_CHECK_VALUE(false, "blkattn: unsupported dtype ", t.scalar_type());
    }
    TORCH_CHECK_VALUE(t.dim() <= 4, "blkattn: at most 4 dimensions");
    d_.data = t.numel() > 0 ? t.data_ptr() : nullptr;
    d_.ndim = (int32_t)t.dim();
    for (int i = 0; i < d_.ndim; ++i) {
      d_.sizes[i] = t.size(i);
      d_.strides[i] = t.stride(i);
    }
    d_.device = t.is_cuda() ? t.get_device() : -1;  // host memory: refused by the library
    given_ = true;
  }
  blkattn_tensor d_{};
  bool given_ = false;
};

const at::Tensor& tensor_of(PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), "blkattn: a tensor is wanted");
  return THPVariable_Unpack(o);
}

at::ScalarType dtype_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  TORCH_CHECK_TYPE(THPDtype_Check(o), "blkattn: a torch dtype is wanted");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// The stream of a call: the given handle (an int), or the current stream of
// t's device.
class CallStream {
 public:
  CallStream(PyObject* o, const at::Tensor& t) {
    const bool given = o != Py_None;
    if (given) {
      void* h = PyLong_AsVoidPtr(o);
      if (h == nullptr && PyErr_Occurred()) throw python_error();
      handle_ = static_cast<cudaStream_t>(h);
    }
    if (!t.is_cuda()) return;  // refused by the library
    const auto current = c10::cuda::getCurrentCUDAStream(t.get_device());
    if (!given) handle_ = current.stream();
    const cudaStream_t plain = handle_ == cudaStreamLegacy ? nullptr : handle_;
    if (plain != current.stream()) current_ = current;
  }
  blkattn_stream_t get() const { return reinterpret_cast<blkattn_stream_t>(handle_); }

  // An output of the call.  On a given stream that is not the current one it
  // is allocated, and filled, on the given one: the current stream's memory
  // may still be in use there, and a fill there is ordered with nothing.  The
  // current stream is recorded as a user: that is where the caller reads it.
  at::Tensor fresh(at::IntArrayRef sizes, const at::TensorOptions& options, bool zeros = false) const {
    if (!current_) return zeros ? at::zeros(sizes, options) : at::empty(sizes, options);
    TORCH_CHECK_VALUE(handle_ != cudaStreamPerThread,
                      "blkattn: torch cannot allocate on the per-thread stream: pass the outputs");
    const auto device = current_->device_index();
    const c10::cuda::CUDAStreamGuard guard(handle_ == cudaStreamLegacy
                                               ? c10::cuda::getDefaultCUDAStream(device)
                                               : c10::cuda::getStreamFromExternal(handle_, device));
    at::Tensor t = zeros ? at::zeros(sizes, options) : at::empty(sizes, options);
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *current_);
    return t;
  }

 private:
  cudaStream_t handle_ = nullptr;
  std::optional<c10::cuda::CUDAStream> current_;  // where it is another one
};

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}
int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

void count(Py_ssize_t have, Py_ssize_t want) {
  TORCH_CHECK_TYPE(have == want, "blkattn: ", want, " arguments are wanted, not ", have);
}

// (status, outputs...) as a tuple that owns them.
PyObject* answer(int status, std::initializer_list<PyObject*> outs) {
  PyObject* t = PyTuple_New(1 + (Py_ssize_t)outs.size());
  if (t == nullptr) throw python_error();
  PyTuple_SET_ITEM(t, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (PyObject* o : outs) PyTuple_SET_ITEM(t, i++, o);
  return t;
}
PyObject* again(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// init(rope, rope_bwd, paged_append, fwd_paged): addresses in libblkattn
PyObject* bind_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (f[i] == nullptr) {
      if (PyErr_Occurred()) throw python_error();
      TORCH_CHECK_VALUE(false, "blkattn: a null entry point");
    }
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(f[0]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(f[1]);
  g_append = reinterpret_cast<decltype(g_append)>(f[2]);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(f[3]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// rope(x, pos, phases, out or None, layout, mscale, out_dtype or None, stream or None, back) -> (status, out)
PyObject* bind_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor& x = tensor_of(a[0]);
  const Desc dx(x), pos(a[1]), ph(a[2]);
  const CallStream stream(a[7], x);
  at::Tensor made;
  if (a[3] == Py_None) made = stream.fresh(x.sizes(), x.options().dtype(dtype_of(a[6], x.scalar_type())));
  const Desc y = made.defined() ? Desc(made) : Desc(a[3]);
  const int st = (a[8] == Py_True ? g_rope_bwd : g_rope)(dx.get(), pos.get(), ph.get(), (int32_t)integer(a[4]),
                                                         (float)number(a[5]), y.get(), stream.get());
  return answer(st, {made.defined() ? THPVariable_Wrap(made) : again(a[3])});
  END_HANDLE_TH_ERRORS
}

// append(k, v, pos, table, k_pages, v_pages, phases or None, layout, mscale, q or None, q_out or None,
//        stream or None) -> (status, q_out: given, made of zeros when q is given without it, or None)
PyObject* bind_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const at::Tensor& k = tensor_of(a[0]);
  const Desc dk(k), v(a[1]), pos(a[2]), table(a[3]), kp(a[4]), vp(a[5]), ph(a[6]), q(a[9]);
  const CallStream stream(a[11], k);
  at::Tensor made;
  if (q.given() && a[10] == Py_None) {  // (zeros: the rows of padding are not written)
    const at::Tensor& tq = tensor_of(a[9]);
    made = stream.fresh(tq.sizes(), tq.options(), true);
  }
  const Desc qo = made.defined() ? Desc(made) : Desc(a[10]);
  const int st = g_append(dk.get(), v.get(), pos.get(), table.get(), kp.get(), vp.get(), ph.get(),
                          (int32_t)integer(a[7]), (float)number(a[8]), q.get(), qo.get(), stream.get());
  return answer(st, {made.defined() ? THPVariable_Wrap(made) : again(a[10])});
  END_HANDLE_TH_ERRORS
}

// fwd(q, k_pages, v_pages, table, seqlens, qpos, tree or None, window, scale or None, out or None, lse or None,
//     out_dtype or None, stream or None) -> (status, out, lse)
PyObject* bind_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const at::Tensor& q = tensor_of(a[0]);
  const Desc dq(q), kp(a[1]), vp(a[2]), table(a[3]), sl(a[4]), qp(a[5]), tree(a[6]);
  TORCH_CHECK_VALUE(q.dim() == 4, "blkattn: q is [B, H_q, T_q, d]");
  const CallStream stream(a[12], q);
  at::Tensor out, lse;
  if (a[9] == Py_None) out = stream.fresh(q.sizes(), q.options().dtype(dtype_of(a[11], at::kFloat)));
  if (a[10] == Py_None) lse = stream.fresh(q.sizes().slice(0, 3), q.options().dtype(at::kFloat));
  const Desc dout = a[9] == Py_None ? Desc(out) : Desc(a[9]);
  const Desc dlse = a[10] == Py_None ? Desc(lse) : Desc(a[10]);
  const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)q.size(3))) : (float)number(a[8]);
  const int st = g_fwd(dq.get(), kp.get(), vp.get(), table.get(), sl.get(), qp.get(), tree.get(), integer(a[7]),
                       scale, dout.get(), dlse.get(), stream.get());
  return answer(st, {a[9] == Py_None ? THPVariable_Wrap(out) : again(a[9]),
                     a[10] == Py_None ? THPVariable_Wrap(lse) : again(a[10])});
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_init)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_append)), METH_FASTCALL, nullptr},
    {"fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_fwd)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_bind", "libblkattn calls on torch tensors", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_bind() { return PyModule_Create(&kModule); }
