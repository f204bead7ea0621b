// Host side of the operators that take a few microseconds on the GPU: argument
// checks, outputs and the C-ABI call in one extension function, on torch's C++
// tensors.  The same in Python (checks, torch.empty, ctypes) takes 12 us for
// one output and 19 us for four, longer than the kernels; this takes 3 to 4 us.
// api.py documents the calls and is their public form.
#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <vector>

#include "../../include/nvfp4moe.h"

namespace {

PyObject* g_error = nullptr;  // binding.Nvfp4Error

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

// Checks a CUDA matrix [T, cols] with contiguous rows; returns its row stride.
int64_t rows(const at::Tensor& t, const char* name, at::ScalarType dtype, int64_t T, int64_t cols, at::Device dev) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.device() == dev && t.scalar_type() == dtype && t.dim() == 2 && t.size(0) == T &&
                        t.size(1) == cols && t.stride(1) == 1,
                    name, " must be a ", dtype, " tensor [", T, ", ", cols, "] on ", dev,
                    " with contiguous rows, not ", t.scalar_type(), " ", t.sizes(), " with strides ", t.strides(),
                    " on ", t.device());
  return T > 1 ? t.stride(0) : cols;
}

// Checks a contiguous CUDA tensor.
void whole(const at::Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, at::Device dev) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.device() == dev && t.scalar_type() == dtype && t.sizes() == shape &&
                        t.is_contiguous(),
                    name, " must be a contiguous ", dtype, " tensor ", shape, " on ", dev, ", not ", t.scalar_type(),
                    " ", t.sizes(), " with strides ", t.strides(), " on ", t.device());
}

// A flag, and a stream's handle (none: the current stream), as Python has them;
// what is neither leaves its Python exception standing.
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
std::optional<cudaStream_t> handle(PyObject* o) {
  if (o == Py_None) return std::nullopt;
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) throw python_error();
  return reinterpret_cast<cudaStream_t>(v);
}

// The device of a call, and its stream: the current one, or the given handle,
// in whose pool the outputs are then allocated.
struct Where {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  at::Device dev;
  cudaStream_t stream;
  Where(const at::Tensor& t, std::optional<cudaStream_t> s) : device(t.device()), dev(t.device()) {
    if (!s) {
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    } else {
      stream = *s;
      guard.reset_stream(c10::cuda::getStreamFromExternal(stream, dev.index()));
    }
  }
  // From the caching allocator, on this stream.
  c10::Storage storage(int64_t bytes, bool resizable) const {
    c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
    return c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                              from->allocate(bytes), from, resizable));
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    return part(storage(c10::multiply_integers(shape) * (int64_t)c10::elementSize(dtype), true), 0, shape, dtype);
  }
  // A contiguous tensor `offset` bytes into a storage.
  static at::Tensor part(c10::Storage s, int64_t offset, at::IntArrayRef shape, at::ScalarType dtype) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        std::move(s), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(dtype));
    if (offset) t.unsafeGetTensorImpl()->set_storage_offset(offset / (int64_t)c10::elementSize(dtype));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
  }
};

// Outputs of one call that live about equally long, parts of one allocation where
// they are small: up to about kShared bytes the kernel takes no longer than the
// host does with an allocation for each (a call with four outputs 5.3 us with an
// allocation each, 4.5 with one for three of them).  The shared
// storage cannot be resized, which would let one part grow into the next.
class Outputs {
 public:
  static constexpr int64_t kShared = 16 << 20, kAlign = 256;
  Outputs(const Where& at, int64_t bytes, int count) : at_(at) {
    if (count > 1 && bytes + count * kAlign <= kShared) pool_ = at.storage(bytes + count * kAlign, false);
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) {
    if (!pool_) return at_.empty(shape, dtype);
    const int64_t at = used_, bytes = c10::multiply_integers(shape) * (int64_t)c10::elementSize(dtype);
    used_ += (bytes + kAlign - 1) / kAlign * kAlign;
    return Where::part(pool_, at, shape, dtype);
  }

 private:
  const Where& at_;
  c10::Storage pool_;
  int64_t used_ = 0;
};

void need_cuda(const at::Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor, not on ", t.device());
}

// The exception of a failed call; nullptr for Python.
PyObject* failed(int status) {
  PyObject* msg = Py_BuildValue("is", status, *nvfp4_last_error() ? nvfp4_last_error() : nvfp4_status_string(status));
  if (msg) PyErr_SetObject(g_error, msg);  // constructed from the tuple
  Py_XDECREF(msg);
  return nullptr;
}

PyObject* wrap(const std::optional<at::Tensor>& t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
  return false;
}

// x, residual | None, weight, eps, normed, quantized, residual_out | None, stream | None
PyObject* add_rms_norm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[2], "weight");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const bool normed = truth(a[4]), quantized = truth(a[5]);
  const std::optional<cudaStream_t> stream = handle(a[7]);
  need_cuda(x, "x");
  TORCH_CHECK_VALUE(x.dim() == 2, "x must have two dimensions, not ", x.dim());
  const Where at(x, stream);
  const int64_t T = x.size(0), H = x.size(1);
  const int64_t ld_x = rows(x, "x", at::kBFloat16, T, H, at.dev);
  const bool f32 = w.scalar_type() == at::kFloat;
  whole(w, "weight", f32 ? at::kFloat : at::kBFloat16, {H}, at.dev);
  const void* r = nullptr;
  int64_t ld_r = 0, ld_o = 0;
  std::optional<at::Tensor> s, y, q, scales;
  if (a[1] != Py_None) {
    const at::Tensor& res = tensor(a[1], "residual");
    ld_r = rows(res, "residual", at::kBFloat16, T, H, at.dev);
    r = res.data_ptr();
  }
  if (a[6] != Py_None) {
    s = tensor(a[6], "residual_out");
    ld_o = rows(*s, "residual_out", at::kBFloat16, T, H, at.dev);
  }
  const bool sum = a[1] != Py_None && !s;
  const int64_t cols = (H + 127) / 128;
  Outputs out_of(at, T * (H * (2 * normed + quantized) + 4 * cols * quantized), normed + 2 * quantized);
  if (sum) {
    s = at.empty({T, H}, at::kBFloat16);
    ld_o = H;
  }
  if (normed) y = out_of.empty({T, H}, at::kBFloat16);
  if (quantized) {
    q = out_of.empty({T, H}, at::kFloat8_e4m3fn);
    scales = out_of.empty({T, cols}, at::kFloat);
  }
  const int rc = nvfp4_add_rmsnorm_fp8(
      x.data_ptr(), ld_x, r, ld_r, w.data_ptr(), f32, T, H, (float)eps, s ? s->data_ptr() : nullptr, ld_o,
      y ? y->data_ptr() : nullptr, q ? q->data_ptr() : nullptr,
      scales ? static_cast<float*>(scales->data_ptr()) : nullptr, at.stream);
  if (rc != NVFP4_OK) return failed(rc);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, wrap(q));
  PyTuple_SET_ITEM(out, 1, wrap(scales));
  PyTuple_SET_ITEM(out, 2, wrap(y));
  PyTuple_SET_ITEM(out, 3, wrap(s));
  return out;
  END_HANDLE_TH_ERRORS
}

// a, a_scale, w, w_scale, f32, out | None, stream | None
PyObject* fp8_linear(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const std::optional<cudaStream_t> stream = handle(p[6]);
  const bool f32 = truth(p[4]);
  const at::Tensor &a = tensor(p[0], "a"), &sa = tensor(p[1], "a_scale"), &w = tensor(p[2], "w"),
                   &sw = tensor(p[3], "w_scale");
  need_cuda(a, "a");
  TORCH_CHECK_VALUE(a.dim() == 2 && w.dim() == 2, "a and w must have two dimensions, not ", a.dim(), " and ", w.dim());
  const Where at(a, stream);
  const int64_t M = a.size(0), K = a.size(1), N = w.size(0), kb = (K + 127) / 128;
  const int64_t ld_a = rows(a, "a", at::kFloat8_e4m3fn, M, K, at.dev);
  whole(w, "w", at::kFloat8_e4m3fn, {N, K}, at.dev);
  whole(sa, "a_scale", at::kFloat, {M, kb}, at.dev);
  whole(sw, "w_scale", at::kFloat, {(N + 127) / 128, kb}, at.dev);
  const at::ScalarType dtype = f32 ? at::kFloat : at::kBFloat16;
  int64_t ld_out = N;
  at::Tensor out;
  if (p[5] != Py_None) {
    out = tensor(p[5], "out");
    ld_out = rows(out, "out", dtype, M, N, at.dev);
  } else {
    out = at.empty({M, N}, dtype);
  }
  const int rc = nvfp4_fp8_linear(a.data_ptr(), ld_a, static_cast<const float*>(sa.data_ptr()), w.data_ptr(),
                                  static_cast<const float*>(sw.data_ptr()), M, N, K, out.data_ptr(), ld_out, f32,
                                  at.stream);
  return rc == NVFP4_OK ? THPVariable_Wrap(out) : failed(rc);
  END_HANDLE_TH_ERRORS
}

// hidden, logits | None, ids | None, ids' weights | None, experts_start, (most T, H, I, E, top_k),
// (w13, w13_sf, w13_gs, w2, w2_sf, w2_gs), gate_limit, up_limit, workspace, out | None, stream | None
PyObject* moe_few_tokens(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 12)) return nullptr;
  const at::Tensor& x = tensor(p[0], "hidden");
  long long start = PyLong_AsLongLong(p[4]), most, H, I, E, k;
  if (start == -1 && PyErr_Occurred()) return nullptr;
  if (!PyArg_ParseTuple(p[5], "LLLLL", &most, &H, &I, &E, &k)) return nullptr;
  TORCH_CHECK_VALUE(PyTuple_Check(p[6]) && PyTuple_GET_SIZE(p[6]) == 6, "six weight tensors expected");
  TORCH_CHECK_VALUE(start >= INT32_MIN && start <= INT32_MAX, "experts_start must be a 32-bit number");
  const double gl = PyFloat_AsDouble(p[7]), ul = PyFloat_AsDouble(p[8]);
  if (PyErr_Occurred()) return nullptr;
  const std::optional<cudaStream_t> stream = handle(p[11]);
  need_cuda(x, "hidden");
  TORCH_CHECK_VALUE(x.dim() == 2, "hidden must have two dimensions, not ", x.dim());
  const Where at(x, stream);
  const int64_t T = x.size(0);
  const int64_t ld = rows(x, "hidden", at::kBFloat16, T, H, at.dev);
  TORCH_CHECK_VALUE(T <= most, T, " tokens; this layer was made for ", most);
  const at::Tensor* w[6];
  static const char* const names[6] = {"w13", "w13_sf", "w13_gs", "w2", "w2_sf", "w2_gs"};
  for (int i = 0; i < 6; ++i) w[i] = &tensor(PyTuple_GET_ITEM(p[6], i), names[i]);
  whole(*w[0], names[0], at::kByte, {E, 2 * I, H / 2}, at.dev);
  whole(*w[3], names[3], at::kByte, {E, H, I / 2}, at.dev);
  const int64_t sizes[6] = {0, E * I * (H / 8), E, 0, E * H * (I / 16), E};
  for (int i : {1, 2, 4, 5})
    TORCH_CHECK_VALUE(w[i]->device() == at.dev && w[i]->numel() == sizes[i] && w[i]->is_contiguous() &&
                          w[i]->scalar_type() == (i % 3 == 1 ? at::kByte : at::kFloat),
                      names[i], " does not belong to this layer");
  const at::Tensor& ws = tensor(p[9], "workspace");
  TORCH_CHECK_VALUE(ws.device() == at.dev, "the layer's workspace is on ", ws.device());
  at::Tensor out;
  if (p[10] != Py_None) {
    out = tensor(p[10], "out");
    whole(out, "out", at::kBFloat16, {T, H}, at.dev);
  }
  const float *g13 = static_cast<const float*>(w[2]->data_ptr()), *g2 = static_cast<const float*>(w[5]->data_ptr());
  int rc;
  if (p[1] != Py_None) {
    const at::Tensor& logits = tensor(p[1], "logits");
    whole(logits, "logits", at::kFloat, {T, E}, at.dev);
    if (!out.defined()) out = at.empty({T, H}, at::kBFloat16);
    rc = nvfp4_moe_few_tokens(x.data_ptr(), ld, static_cast<const float*>(logits.data_ptr()), T, H, I, (int)E, (int)k,
                              w[0]->data_ptr(), w[1]->data_ptr(), g13, w[3]->data_ptr(), w[4]->data_ptr(), g2,
                              (float)gl, (float)ul, ws.data_ptr(), ws.nbytes(), out.data_ptr(), at.stream);
  } else {
    const at::Tensor &ids = tensor(p[2], "topk_ids"), &pw = tensor(p[3], "topk_weights");
    whole(ids, "topk_ids", at::kInt, {T, k}, at.dev);
    whole(pw, "topk_weights", at::kFloat, {T, k}, at.dev);
    if (!out.defined()) out = at.empty({T, H}, at::kBFloat16);
    rc = nvfp4_moe_few_tokens_routed(x.data_ptr(), ld, static_cast<const int32_t*>(ids.data_ptr()),
                                     static_cast<const float*>(pw.data_ptr()), (int32_t)start, T, H, I, (int)E,
                                     (int)k, w[0]->data_ptr(), w[1]->data_ptr(), g13, w[3]->data_ptr(),
                                     w[4]->data_ptr(), g2, (float)gl, (float)ul, ws.data_ptr(), ws.nbytes(),
                                     out.data_ptr(), at.stream);
  }
  return rc == NVFP4_OK ? THPVariable_Wrap(out) : failed(rc);
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define CALL(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(add_rms_norm_fp8), CALL(fp8_linear), CALL(moe_few_tokens),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
