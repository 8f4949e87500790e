// Argument marshalling of the calls a decode step makes several times per layer
// (pad_qk_norm_rope, pad_append_kv, pad_decode_shared): torch tensors to
// pad_tensor descriptors, outputs allocated, one library call.  From Python a
// descriptor costs a microsecond and a call 15, which is more than the kernels of a
// small step; here a call costs about as much as its launch.  Measured, norm and
// rotation of 16 tokens: 3.2 us for the C call alone (its launch 2 of them).
//
// A function returns its outputs, or the status of a failed call as an int.  The
// library's entry points are handed over by address (bind), so that this module
// uses the libpad.so that the package loaded.
#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pad.h"

namespace {

decltype(&pad_qk_norm_rope) g_norm_rope = nullptr;
decltype(&pad_append_kv) g_append = nullptr;
decltype(&pad_decode_shared) g_shared = nullptr;

// torch gives a tensor without elements no address, and the library takes null for no
// tensor (or refuses it): any other will do, as nothing reads it.
void *address_of(const at::Tensor &t) { return t.numel() == 0 ? reinterpret_cast<void *>(256) : t.data_ptr(); }

// The descriptor of an optional tensor argument; address() is null for None.
class Desc {
 public:
  Desc(PyObject *o, const char *name) {
    if (o == Py_None) return;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor or None");
    set(THPVariable_Unpack(o), name);
  }
  Desc(const at::Tensor &t, const char *name) {
    if (t.defined()) set(t, name);
  }
  pad_tensor *address() { return some_ ? &d_ : nullptr; }

 private:
  void set(const at::Tensor &t, const char *name) {
    some_ = true;
    d_.data = address_of(t);
    switch (t.scalar_type()) {
      case at::kBFloat16: d_.dtype = PAD_BF16; break;
      case at::kFloat: d_.dtype = PAD_F32; break;
      case at::kInt: d_.dtype = PAD_I32; break;
      case at::kFloat8_e4m3fn: d_.dtype = PAD_FP8_E4M3; break;
      default: TORCH_CHECK_TYPE(false, name, ": unsupported dtype ", t.scalar_type());
    }
    TORCH_CHECK_VALUE(t.dim() <= 4, name, ": at most 4 dims, got ", t.dim());
    d_.ndim = (int32_t)t.dim();
    for (int i = 0; i < d_.ndim; ++i) {
      d_.shape[i] = t.size(i);
      d_.stride[i] = t.stride(i);
    }
  }
  pad_tensor d_{};
  bool some_ = false;
};

const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  const at::Tensor &t = THPVariable_Unpack(o);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor, is on ", t.device());
  return t;
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
  return at::detail::empty_cuda(sizes, type, like.device(), c10::nullopt);  // (past the dispatcher: half its time)
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
int truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
void *handle(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw python_error();
  return p;
}

// The stream of a call: torch's current one of the tensor's device (None), or one given
// beside it.  torch's allocator gives a block out again in the order of the stream that it
// was allocated on, so a stream beside that has to be made known to it: outputs come from
// the call's stream and are marked for the current one, where the caller goes on with
// them; the caller's tensors are marked for the call's.
class On {
 public:
  On(PyObject *o, const at::Tensor &t)
      : current_(c10::cuda::getCurrentCUDAStream(t.get_device())), call_(current_), handle_(current_.stream()) {
    if (o == Py_None) return;
    handle_ = handle(o);
    cudaStream_t s = static_cast<cudaStream_t>(handle_);
    if (s == cudaStreamLegacy) s = nullptr;
    // (one handle for a stream in every thread: an event that the allocator records on
    // it when it frees a block may be another thread's)
    unknown_ = s == cudaStreamPerThread;
    beside_ = !unknown_ && s != current_.stream();
    if (beside_) call_ = c10::cuda::getStreamFromExternal(s, t.get_device());
  }
  void *stream() const { return handle_; }
  at::Tensor allocate(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) const {
    TORCH_CHECK_VALUE(!unknown_, "on cudaStreamPerThread the outputs must be given: torch's allocator cannot follow it");
    if (!beside_) return empty(sizes, type, like);
    c10::cuda::CUDAStreamGuard guard(call_);
    at::Tensor t = empty(sizes, type, like);
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current_);
    return t;
  }
  // An output: the caller's tensor, or a contiguous one of the shape and type of `like`.
  at::Tensor output(PyObject *o, const at::Tensor &like, const char *name) const {
    return o == Py_None ? allocate(like.sizes(), like.scalar_type(), like) : cuda_tensor(o, name);
  }
  // The call's arguments, once it is launched.
  void used(PyObject *const *a, Py_ssize_t n) const {
    if (!beside_) return;
    for (Py_ssize_t i = 0; i < n; ++i)
      if (THPVariable_Check(a[i])) c10::cuda::CUDACachingAllocator::recordStream(THPVariable_Unpack(a[i]).storage().data_ptr(), call_);
  }

 private:
  c10::cuda::CUDAStream current_, call_;
  void *handle_;
  bool beside_ = false, unknown_ = false;
};

void expect(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <class F>
pad_status without_gil(F &&call) {
  PyThreadState *s = PyEval_SaveThread();
  const pad_status st = call();
  PyEval_RestoreThread(s);
  return st;
}

PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 3);
  g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(handle(a[0]));
  g_append = reinterpret_cast<decltype(g_append)>(handle(a[1]));
  g_shared = reinterpret_cast<decltype(g_shared)>(handle(a[2]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, q_out, k_out, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 11);
  const at::Tensor &q = cuda_tensor(a[0], "q");
  c10::cuda::CUDAGuard device(q.device());
  const On on(a[10], q);
  at::Tensor q_out = on.output(a[8], q, "q_out"), k_out;
  if (a[1] != Py_None) k_out = on.output(a[9], cuda_tensor(a[1], "k"), "k_out");
  else if (a[9] != Py_None) k_out = cuda_tensor(a[9], "k_out");
  Desc dq(a[0], "q"), dk(a[1], "k"), dqw(a[2], "q_weight"), dkw(a[3], "k_weight"), dp(a[4], "positions"),
      df(a[5], "inv_freq"), dqo(q_out, "q_out"), dko(k_out, "k_out");
  const float eps = number(a[6]);
  const int inter = truth(a[7]);
  const pad_status st = without_gil([&] {
    return g_norm_rope(dq.address(), dk.address(), dqw.address(), dkw.address(), eps, dp.address(), df.address(), inter,
                       dqo.address(), dko.address(), on.stream());
  });
  if (st != PAD_OK) return PyLong_FromLong(st);
  on.used(a, n);
  PyObject *x = wrap(q_out), *y = wrap(k_out);
  PyObject *r = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
  END_HANDLE_TH_ERRORS
}

// k, v, positions, block_tables, k_cache, v_cache, seq_ids, inv_freq, interleaved, k_weight, eps, q, q_weight, q_out,
// k_scale, v_scale, stream
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 17);
  const at::Tensor &k = cuda_tensor(a[0], "k");
  c10::cuda::CUDAGuard device(k.device());
  const On on(a[16], k);
  TORCH_CHECK_VALUE(a[11] != Py_None || a[13] == Py_None, "q_out without q");
  at::Tensor q_out;
  if (a[11] != Py_None) q_out = on.output(a[13], cuda_tensor(a[11], "q"), "q_out");
  Desc dk(a[0], "k"), dv(a[1], "v"), dp(a[2], "positions"), dt(a[3], "block_tables"), dkc(a[4], "k_cache"),
      dvc(a[5], "v_cache"), ds(a[6], "seq_ids"), df(a[7], "inv_freq"), dkw(a[9], "k_weight"), dq(a[11], "q"),
      dqw(a[12], "q_weight"), dqo(q_out, "q_out");
  pad_append_options o{};
  o.inv_freq = df.address();
  o.interleaved = truth(a[8]);
  o.k_weight = dkw.address();
  o.eps = number(a[10]);
  o.q = dq.address();
  o.q_weight = dqw.address();
  o.q_out = dqo.address();
  o.k_scale = number(a[14]);
  o.v_scale = number(a[15]);
  const pad_status st = without_gil([&] {
    return g_append(dk.address(), dv.address(), dp.address(), ds.address(), dt.address(), &o, dkc.address(),
                    dvc.address(), on.stream());
  });
  if (st != PAD_OK) return PyLong_FromLong(st);
  on.used(a, n);
  return wrap(q_out);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, shared_table, block_tables, seq_lens, scale, out, lse (tensor, None or True), sinks, k_scale,
// v_scale, workspace, stream
PyObject *decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 14);
  const at::Tensor &q = cuda_tensor(a[0], "q");
  c10::cuda::CUDAGuard device(q.device());
  const On on(a[13], q);
  at::Tensor out = on.output(a[7], q, "out"), lse;
  if (a[8] == Py_True) {
    TORCH_CHECK_VALUE(q.dim() >= 2, "q must be [B, Hq, D]");
    lse = on.allocate({q.size(0), q.size(1)}, at::kFloat, q);
  } else if (a[8] != Py_None && a[8] != Py_False) {
    lse = cuda_tensor(a[8], "lse");
  }
  Desc dq(a[0], "q"), dk(a[1], "k_cache"), dv(a[2], "v_cache"), dsh(a[3], "shared_table"), dt(a[4], "block_tables"),
      dl(a[5], "seq_lens"), dout(out, "out"), dlse(lse, "lse"), dsk(a[9], "sinks");
  const float scale = number(a[6]);
  pad_decode_options o{};
  o.sinks = dsk.address();
  o.k_scale = number(a[10]);
  o.v_scale = number(a[11]);
  void *ws = nullptr;
  size_t ws_bytes = 0;
  if (a[12] != Py_None) {
    const at::Tensor &w = cuda_tensor(a[12], "workspace");
    TORCH_CHECK_VALUE(w.device() == q.device() && w.is_contiguous(),
                      "workspace must be a contiguous tensor on q's device");
    ws = address_of(w);
    ws_bytes = w.numel() * w.element_size();
  }
  const pad_status st = without_gil([&] {
    return g_shared(dq.address(), dk.address(), dv.address(), dsh.address(), dt.address(), dl.address(), scale, &o,
                    dout.address(), dlse.address(), ws, ws_bytes, on.stream());
  });
  if (st != PAD_OK) return PyLong_FromLong(st);
  on.used(a, n);
  PyObject *x = wrap(out), *y = wrap(lse);
  PyObject *r = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&bind)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&qk_norm_rope)), METH_FASTCALL, nullptr},
    {"append_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&append_kv)), METH_FASTCALL, nullptr},
    {"decode_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&decode_shared)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pad_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pad_torch(void) { return PyModule_Create(&module); }
