// binding.cpp -- the Python calls of the entry points around the loss
// (grpo_token_logps, grpo_token_logps_grad, grpo_clip_grad_norm): argument
// checks, output allocation and the C call, natively.
//
// Argument marshalling only, as in the package's ctypes calls.  These three
// are called once a generated token or with hundreds of tensors, where the
// checks and allocations in Python cost more than the kernels (0.9 us a tensor
// of a clipping call there, 47 ns here with the launches' tables).
//
// Every function takes its arguments by position, works on the current stream
// of the tensors' device, raises ValueError for what the C ABI cannot see
// (devices, dtypes, shapes), and returns either its results or the C status as
// an int.  No C++ exception leaves a function.
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/grpo.h"

namespace {

// What becomes a ValueError.
struct Refused : std::invalid_argument {
  using std::invalid_argument::invalid_argument;
};

#define GRPO_TRY try {
#define GRPO_CATCH                                    \
  }                                                   \
  catch (const Refused& e) {                          \
    PyErr_SetString(PyExc_ValueError, e.what());      \
    return nullptr;                                   \
  }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GRPO_F32;
    case at::kBFloat16: return GRPO_BF16;
    case at::kHalf: return GRPO_F16;
    default: return -1;
  }
}

// Logits [B, T, V] or [N, V] whose rows hold adjacent elements.
struct Rows {
  int64_t B, T, V, sb, st;
  int dt;
  Rows(const at::Tensor& x, const char* name) {
    const std::string n(name);
    dt = dtype_code(x.scalar_type());
    if (dt < 0) throw Refused("unsupported " + n + " dtype " + c10::toString(x.scalar_type()));
    if (!x.is_cuda()) throw Refused(n + " must be a CUDA tensor");
    int64_t sv;
    if (x.dim() == 3) {
      B = x.size(0); T = x.size(1); V = x.size(2);
      sb = x.stride(0); st = x.stride(1); sv = x.stride(2);
    } else if (x.dim() == 2) {
      B = x.size(0); T = 1; V = x.size(1);
      sb = x.stride(0); st = 0; sv = x.stride(1);
    } else {
      throw Refused(n + " must be [B, T, V] or [N, V]");
    }
    if (sv != 1 && V > 1) throw Refused("the logits of a row of " + n + " must be adjacent (stride 1)");
  }
};

// The pointer of a contiguous per-token tensor (nullptr for None): dtype t,
// or bool / uint8 for a mask; `extra` sizes before the logits' leading ones.
void* token(PyObject* o, const char* name, const at::Tensor& x, at::ScalarType t, int extra = 0) {
  if (o == Py_None) return nullptr;
  const at::Tensor& v = tensor(o, name);
  const int lead = (int)x.dim() - 1;
  const bool mask = t == at::kByte;
  bool ok = (v.scalar_type() == t || (mask && v.scalar_type() == at::kBool)) &&
            v.dim() == lead + (extra ? 1 : 0) && v.device() == x.device() && v.is_contiguous();
  if (ok && extra) ok = v.size(0) == extra;
  for (int i = 0; ok && i < lead; ++i) ok = v.size(i + (extra ? 1 : 0)) == x.size(i);
  if (!ok)
    throw Refused(std::string(name) + " must be a contiguous " +
                  (mask ? "bool or uint8" : c10::toString(t)) + " tensor" +
                  (extra ? " [2, ...]" : "") +
                  " of the logits' leading shape on their device, got " +
                  c10::toString(v.scalar_type()) + " " + c10::str(v.sizes()) + " on " +
                  v.device().str());
  return v.data_ptr();
}

void* status_word(PyObject* o, const at::Tensor& x) {
  if (o == Py_None) return nullptr;
  const at::Tensor& v = tensor(o, "status");
  if (v.device() != x.device() || !v.is_contiguous() || v.nbytes() < 256)
    throw Refused("status must be a status_buffer() on the device of the logits");
  return v.data_ptr();
}

void put(PyObject* dict, const char* name, const at::Tensor& t) {
  PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  if (!o) throw python_error();
  const int rc = PyDict_SetItemString(dict, name, o);
  Py_DECREF(o);
  if (rc != 0) throw python_error();
}

// A tensor of the caller's was written through its pointer: autograd has to see
// that a value it saved is gone.  (Inference tensors count no versions.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

PyObject* want_args(Py_ssize_t n, Py_ssize_t want) {
  PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
  return nullptr;
}

// token_logps(logits, action_ids, completion_mask, temperature, top_k,
//             want_entropy, want_stats, status) -> dict or status code
PyObject* token_logps(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GRPO_TRY
  if (n != 8) return want_args(n, 8);
  const at::Tensor& x = tensor(a[0], "logits");
  const Rows r(x, "logits");
  void* ids = token(a[1], "action_ids", x, at::kLong);
  void* mask = token(a[2], "completion_mask", x, at::kByte);
  const double temperature = number(a[3]);
  const long long k = PyLong_AsLongLong(a[4]);
  if (k == -1 && PyErr_Occurred()) return nullptr;
  const bool want_entropy = flag(a[5]), want_stats = flag(a[6]);
  void* status = status_word(a[7], x);
  const c10::cuda::CUDAGuard guard(x.device());
  const auto f32 = at::TensorOptions().dtype(at::kFloat).device(x.device());
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  at::Tensor logps, entropy, stats, top_ids, top_logps;
  if (a[1] != Py_None) logps = at::empty(lead, f32);
  if (want_entropy) entropy = at::empty(lead, f32);
  if (want_stats) {
    c10::SmallVector<int64_t, 4> s{2};
    s.append(lead.begin(), lead.end());
    stats = at::empty(s, f32);
  }
  if (k > 0 && k <= GRPO_MAX_TOP_K) {  // (others are refused below)
    c10::SmallVector<int64_t, 4> s(lead.begin(), lead.end());
    s.push_back(k);
    top_ids = at::empty(s, f32.dtype(at::kLong));
    top_logps = at::empty(s, f32);
  }
  auto at_ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  grpo_status_t rc;
  const auto stream = c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
  const int32_t k32 = k < 0 || k > GRPO_MAX_TOP_K ? -1 : (int32_t)k;
  Py_BEGIN_ALLOW_THREADS
  rc = grpo_token_logps(x.data_ptr(), (grpo_dtype_t)r.dt, r.B, r.T, r.V, r.sb, r.st,
                        (const int64_t*)ids, (const uint8_t*)mask, (float)temperature, k32,
                        (float*)at_ptr(logps), (float*)at_ptr(entropy), (float*)at_ptr(stats),
                        (int64_t*)at_ptr(top_ids), (float*)at_ptr(top_logps), status, stream);
  Py_END_ALLOW_THREADS
  if (rc != GRPO_OK) return PyLong_FromLong((long)rc);
  THPObjectPtr out(PyDict_New());
  if (!out) return nullptr;
  put(out, "logps", logps);
  put(out, "entropy", entropy);
  put(out, "stats", stats);
  put(out, "top_ids", top_ids);
  put(out, "top_logps", top_logps);
  return out.release();
  GRPO_CATCH
  END_HANDLE_TH_ERRORS
}

// token_logps_grad(logits, action_ids, completion_mask, stats, grad_logps,
//                  entropy, grad_entropy, temperature, grad, skip_masked,
//                  status) -> gradient or status code
PyObject* token_logps_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  GRPO_TRY
  if (n != 11) return want_args(n, 11);
  const at::Tensor& x = tensor(a[0], "logits");
  const Rows r(x, "logits");
  void* ids = token(a[1], "action_ids", x, at::kLong);
  void* mask = token(a[2], "completion_mask", x, at::kByte);
  if (a[3] == Py_None) throw Refused("stats (of grpo_token_logps, with want_stats) is required");
  void* stats = token(a[3], "stats", x, at::kFloat, 2);
  void* dlogp = token(a[4], "grad_logps", x, at::kFloat);
  void* ent = token(a[5], "entropy", x, at::kFloat);
  void* dent = token(a[6], "grad_entropy", x, at::kFloat);
  const double temperature = number(a[7]);
  const uint32_t flags = flag(a[9]) ? GRPO_SKIP_MASKED_GRAD_ROWS : 0u;
  void* status = status_word(a[10], x);
  const c10::cuda::CUDAGuard guard(x.device());
  at::Tensor grad;
  if (a[8] == Py_None) {
    grad = at::empty(x.sizes(), x.options());
  } else {
    grad = tensor(a[8], "grad");
    if (grad.sizes() != x.sizes() || grad.scalar_type() != x.scalar_type() ||
        grad.device() != x.device())
      throw Refused("grad must have the shape, dtype and device of logits");
  }
  const Rows g(grad, "grad");
  grpo_status_t rc;
  const auto stream = c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
  Py_BEGIN_ALLOW_THREADS
  rc = grpo_token_logps_grad(x.data_ptr(), (grpo_dtype_t)r.dt, r.B, r.T, r.V, r.sb, r.st,
                             (const int64_t*)ids, (const uint8_t*)mask, (const float*)stats,
                             (const float*)ent, (const float*)dlogp, (const float*)dent,
                             (float)temperature, grad.data_ptr(), g.sb, g.st, flags, status,
                             stream);
  Py_END_ALLOW_THREADS
  if (rc != GRPO_OK) return PyLong_FromLong((long)rc);
  if (a[8] != Py_None) written(grad);
  return THPVariable_Wrap(grad);
  GRPO_CATCH
  END_HANDLE_TH_ERRORS
}

// clip_grad_norm(tensors: tuple, max_norm, eps, scale, out: tuple or None,
//                norm_only, workspace) -> dict or status code
// Tuples hold their tensors while the call runs without the GIL (another thread
// may change a list); references of its own to each of 291 tensors cost 4 us.
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  GRPO_TRY
  if (nargs != 7) return want_args(nargs, 7);
  if (!PyTuple_Check(a[0]) || (a[4] != Py_None && !PyTuple_Check(a[4]))) {
    PyErr_SetString(PyExc_TypeError, "tensors and out are tuples");
    return nullptr;
  }
  const int64_t n = PyTuple_GET_SIZE(a[0]);
  const bool outs = a[4] != Py_None, norm_only = flag(a[5]);
  const double max_norm = number(a[1]), eps = number(a[2]), scale = number(a[3]);
  if (outs && norm_only) throw Refused("norm_only writes nothing: out must be None");
  if (outs && PyTuple_GET_SIZE(a[4]) != n)
    throw Refused("out must hold one tensor for each of tensors");
  std::vector<const void*> in(n), seen;
  std::vector<void*> to(outs ? n : 0);
  std::vector<int64_t> numel(n);
  std::vector<int32_t> dtype(n);
  seen.reserve(n);
  c10::Device dev(at::kCUDA, n > 0 ? (c10::DeviceIndex)0 : c10::cuda::current_device());
  for (int64_t i = 0; i < n; ++i) {
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(a[0], i), "a gradient");
    if (!t.is_cuda()) throw Refused("tensors must be CUDA tensors");
    if (i == 0) dev = t.device();
    if (t.device() != dev) throw Refused("every tensor must be on one device");
    dtype[i] = dtype_code(t.scalar_type());
    if (dtype[i] < 0)
      throw Refused(std::string("unsupported gradient dtype ") + c10::toString(t.scalar_type()));
    if (!t.is_contiguous() && !t.is_non_overlapping_and_dense())
      throw Refused("tensors must be dense (no gaps between elements)");
    in[i] = t.data_ptr();
    numel[i] = t.numel();
    if (numel[i] > 0) seen.push_back(in[i]);
    if (!outs) continue;
    const at::Tensor& o = tensor(PyTuple_GET_ITEM(a[4], i), "an output");
    if (o.device() != dev || o.scalar_type() != t.scalar_type() || o.numel() != t.numel())
      throw Refused("out must hold a tensor of the same size and dtype, on the same device, for "
                    "each of tensors");
    // element i of the memory of one belongs to element i of the other
    if (!(t.is_contiguous() && o.is_contiguous()) &&
        !(t.sizes() == o.sizes() && t.strides() == o.strides()))
      throw Refused("out must be contiguous as tensors are, or have their strides");
    to[i] = o.data_ptr();
  }
  std::sort(seen.begin(), seen.end());
  if (std::adjacent_find(seen.begin(), seen.end()) != seen.end())
    throw Refused("a tensor is given twice");
  const c10::cuda::CUDAGuard guard(dev);
  const auto f32 = at::TensorOptions().dtype(at::kFloat).device(dev);
  // The workspace goes back to the allocator with this call: the results, which
  // a caller may keep, are a tensor of two numbers.
  size_t need = 0;
  void* ws = nullptr;
  c10::DataPtr own;
  if (a[6] != Py_None) {
    const at::Tensor& given = tensor(a[6], "workspace");
    if (given.device() != dev || !given.is_contiguous())
      throw Refused("workspace must be a contiguous tensor on the device of tensors");
    ws = given.data_ptr();
    need = given.nbytes();
  } else {
    need = grpo_clip_workspace_size(n);
    own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
    ws = own.get();
  }
  // (a fresh tensor and its two halves: nothing for autograd's dispatch keys)
  const at::AutoDispatchBelowADInplaceOrView below;
  const at::Tensor out2 = at::empty({2}, f32);
  grpo_status_t rc;
  const auto stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  Py_BEGIN_ALLOW_THREADS
  rc = grpo_clip_grad_norm(in.data(), outs ? to.data() : nullptr, numel.data(), dtype.data(), n,
                           (float)max_norm, (float)eps, (float)scale,
                           norm_only ? GRPO_CLIP_NORM_ONLY : 0u, (float*)out2.data_ptr(), ws, need,
                           stream);
  Py_END_ALLOW_THREADS
  if (rc != GRPO_OK) return PyLong_FromLong((long)rc);
  if (!norm_only)
    for (int64_t i = 0; i < n; ++i)
      written(THPVariable_Unpack(PyTuple_GET_ITEM(outs ? a[4] : a[0], i)));
  THPObjectPtr out(PyDict_New());
  if (!out) return nullptr;
  put(out, "norm", out2.select(0, 0));
  put(out, "factor", out2.select(0, 1));
  return out.release();
  GRPO_CATCH
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"token_logps", (PyCFunction)(void (*)(void))token_logps, METH_FASTCALL, nullptr},
    {"token_logps_grad", (PyCFunction)(void (*)(void))token_logps_grad, METH_FASTCALL, nullptr},
    {"clip_grad_norm", (PyCFunction)(void (*)(void))clip_grad_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
