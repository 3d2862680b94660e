// Argument marshalling of the serving-step operators (rope, head norms, paged
// append, attention over pages) for torch tensors: descriptors straight from the
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
decltype(&blkattn_qk_norm_rope) g_norm;
decltype(&blkattn_qk_norm_rope_bwd) g_norm_bwd;
decltype(&blkattn_paged_append_q8) g_append_q8;
decltype(&blkattn_paged_read_q8) g_read_q8;
decltype(&blkattn_fwd_paged_q8) g_fwd_q8;

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
      case at::kFloat8_e4m3fn: d_.dtype = BLKATTN_E4M3; break;
      case at::kFloat8_e8m0fnu: d_.dtype = BLKATTN_E8M0; break;
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

// init(rope, rope_bwd, paged_append, fwd_paged, qk_norm_rope, qk_norm_rope_bwd, paged_append_q8, paged_read_q8,
//      fwd_paged_q8): addresses in libblkattn
PyObject* bind_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int kEntries = 9;
  count(n, kEntries);
  void* f[kEntries];
  for (int i = 0; i < kEntries; ++i) {
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
  g_norm = reinterpret_cast<decltype(g_norm)>(f[4]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(f[5]);
  g_append_q8 = reinterpret_cast<decltype(g_append_q8)>(f[6]);
  g_read_q8 = reinterpret_cast<decltype(g_read_q8)>(f[7]);
  g_fwd_q8 = reinterpret_cast<decltype(g_fwd_q8)>(f[8]);
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

// An output argument: the given object, or, for None, a fresh tensor.
class Out {
 public:
  Out(PyObject* given, const CallStream& stream, at::IntArrayRef sizes, const at::TensorOptions& options, bool zeros = false)
      : given_(given), d_(given == Py_None ? Desc(made_ = stream.fresh(sizes, options, zeros)) : Desc(given)) {}
  explicit Out(PyObject* none) : given_(none), d_(none) {}  // an output that the call does without
  const blkattn_tensor* get() const { return d_.get(); }
  PyObject* object() const { return made_.defined() ? THPVariable_Wrap(made_) : again(given_); }

 private:
  at::Tensor made_;
  PyObject* given_;
  Desc d_;
};

// norm(q, k or None, wq, wk or None, pos, phases or None, layout, mscale, eps, out_dtype or None, q_out or None,
//      k_out or None, stream or None) -> (status, q_out, k_out)
PyObject* bind_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const at::Tensor& q = tensor_of(a[0]);
  const Desc dq(q), dk(a[1]), wq(a[2]), wk(a[3]), pos(a[4]), ph(a[5]);
  const CallStream stream(a[12], q);
  const auto options = q.options().dtype(dtype_of(a[9], q.scalar_type()));
  const Out qo(a[10], stream, q.sizes(), options);
  const Out ko = a[1] == Py_None ? Out(a[11]) : Out(a[11], stream, tensor_of(a[1]).sizes(), options);
  const int st = g_norm(dq.get(), wq.get(), dk.get(), wk.get(), pos.get(), ph.get(), (int32_t)integer(a[6]),
                        (float)number(a[7]), (float)number(a[8]), qo.get(), ko.get(), stream.get());
  return answer(st, {qo.object(), ko.object()});
  END_HANDLE_TH_ERRORS
}

// norm_bwd(dq_out, dk_out or None, q, k or None, wq, wk or None, pos, phases or None, layout, mscale, eps,
//          out_dtype or None, dq or None, dk or None, stream or None) -> (status, dq, dk, dq_weight, dk_weight)
PyObject* bind_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const at::Tensor& q = tensor_of(a[2]);
  const at::Tensor& w = tensor_of(a[4]);
  const Desc gq(a[0]), gk(a[1]), dq(q), dk(a[3]), wq(a[4]), wk(a[5]), pos(a[6]), ph(a[7]);
  const CallStream stream(a[14], q);
  const auto options = q.options().dtype(dtype_of(a[11], q.scalar_type()));
  const auto sums = q.options().dtype(at::kFloat);
  const bool two = a[3] != Py_None;
  const Out oq(a[12], stream, q.sizes(), options);
  const Out ok = two ? Out(a[13], stream, tensor_of(a[3]).sizes(), options) : Out(a[13]);
  const Out owq(Py_None, stream, w.sizes(), sums);
  const Out owk = two ? Out(Py_None, stream, w.sizes(), sums) : Out(Py_None);
  const int st = g_norm_bwd(gq.get(), gk.get(), dq.get(), wq.get(), dk.get(), wk.get(), pos.get(), ph.get(),
                            (int32_t)integer(a[8]), (float)number(a[9]), (float)number(a[10]), oq.get(), ok.get(),
                            owq.get(), owk.get(), stream.get());
  return answer(st, {oq.object(), ok.object(), owq.object(), owk.object()});
  END_HANDLE_TH_ERRORS
}

// append_q8(k, v, pos, table, k_pages, v_pages, k_scales, v_scales, phases or None, layout, mscale, k_weight or None,
//           q_weight or None, eps, q or None, q_out or None, stream or None) -> (status, q_out, as append)
PyObject* bind_append_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17);
  const at::Tensor& k = tensor_of(a[0]);
  const Desc dk(k), v(a[1]), pos(a[2]), table(a[3]), kp(a[4]), vp(a[5]), ks(a[6]), vs(a[7]), ph(a[8]), wk(a[11]),
      wq(a[12]), q(a[14]);
  const CallStream stream(a[16], k);
  // (zeros: the rows of padding are not written)
  const Out qo = q.given() ? Out(a[15], stream, tensor_of(a[14]).sizes(), tensor_of(a[14]).options(), true) : Out(a[15]);
  const int st = g_append_q8(dk.get(), v.get(), pos.get(), table.get(), kp.get(), vp.get(), ks.get(), vs.get(),
                             wk.get(), (float)number(a[13]), ph.get(), (int32_t)integer(a[9]), (float)number(a[10]),
                             q.get(), wq.get(), qo.get(), stream.get());
  return answer(st, {qo.object()});
  END_HANDLE_TH_ERRORS
}

// read_q8(pos, table, k_pages, v_pages, k_scales, v_scales, out_dtype or None, k_out or None, v_out or None,
//         stream or None) -> (status, k_out, v_out)
PyObject* bind_read_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const at::Tensor& kp = tensor_of(a[2]);
  const at::Tensor& tp = tensor_of(a[0]);
  const Desc pos(tp), table(a[1]), dk(kp), vp(a[3]), ks(a[4]), vs(a[5]);
  TORCH_CHECK_VALUE(kp.dim() == 4 && tp.dim() == 2, "blkattn: pos is [B, T], the pools [N, H_kv, P, d]");
  const CallStream stream(a[9], kp);
  const int64_t sizes[4] = {tp.size(0), kp.size(1), tp.size(1), kp.size(3)};
  const auto options = kp.options().dtype(dtype_of(a[6], at::kBFloat16));
  const Out ko(a[7], stream, sizes, options), vo(a[8], stream, sizes, options);
  const int st = g_read_q8(pos.get(), table.get(), dk.get(), vp.get(), ks.get(), vs.get(), ko.get(), vo.get(),
                           stream.get());
  return answer(st, {ko.object(), vo.object()});
  END_HANDLE_TH_ERRORS
}

// fwd_q8(q, k_pages, v_pages, k_scales, v_scales, table, seqlens, qpos, tree or None, window, scale or None,
//        out or None, lse or None, out_dtype or None, stream or None) -> (status, out, lse)
PyObject* bind_fwd_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const at::Tensor& q = tensor_of(a[0]);
  const Desc dq(q), kp(a[1]), vp(a[2]), ks(a[3]), vs(a[4]), table(a[5]), sl(a[6]), qp(a[7]), tree(a[8]);
  TORCH_CHECK_VALUE(q.dim() == 4, "blkattn: q is [B, H_q, T_q, d]");
  const CallStream stream(a[14], q);
  const Out out(a[11], stream, q.sizes(), q.options().dtype(dtype_of(a[13], at::kFloat)));
  const Out lse(a[12], stream, q.sizes().slice(0, 3), q.options().dtype(at::kFloat));
  const float scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)q.size(3))) : (float)number(a[10]);
  const int st = g_fwd_q8(dq.get(), kp.get(), vp.get(), ks.get(), vs.get(), table.get(), sl.get(), qp.get(), tree.get(),
                          integer(a[9]), scale, out.get(), lse.get(), stream.get());
  return answer(st, {out.object(), lse.object()});
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_init)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_append)), METH_FASTCALL, nullptr},
    {"fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_fwd)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_norm)), METH_FASTCALL, nullptr},
    {"norm_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_norm_bwd)), METH_FASTCALL, nullptr},
    {"append_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_append_q8)), METH_FASTCALL, nullptr},
    {"read_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_read_q8)), METH_FASTCALL, nullptr},
    {"fwd_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_fwd_q8)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_bind", "libblkattn calls on torch tensors", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_bind() { return PyModule_Create(&kModule); }
