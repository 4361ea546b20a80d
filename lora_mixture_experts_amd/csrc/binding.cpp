// Compiled half of the Python binding for the operators whose kernels take a few microseconds
// (moe_lora_route, moe_lora_linear): checks of torch tensors, outputs and workspaces from torch's
// allocator, torch's current stream, one call of the C ABI. As attribute reads and ctypes conversions in
// Python the same took 6 us of a 10 us call; here 1 us.
//
// Every function returns its output tensors, or the int code of a call that the C ABI refused.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "byte_ranges.h"
#include "moelora.h"

namespace {

using at::Tensor;
using moelora::Bytes;
using moelora::dense_bytes;
using moelora::overlap;

struct Refused {};  // a Python exception is set
PyObject* out_of_memory = nullptr;  // torch.OutOfMemoryError

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name, const char* more = "") {
  PyErr_Format(type, format, name, more);
  throw Refused{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    case at::kBool: return "torch.bool";
    case at::kInt: return "torch.int32";
    default: return "another type";
  }
}

const Tensor* tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor%s", name);
  return &THPVariable_Unpack(o);
}

void check(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", name, type_name(type));
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s has another shape than the other arguments ask for%s", name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a GPU%s", name);
  if (t.get_device() != device) refuse(PyExc_ValueError, "%s is on another GPU than the first argument%s", name);
}

// Pointer of a contiguous tensor, null for None.
void* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = *tensor_of(o, name);
  check(t, name, type, shape, device);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", name);
  return t.data_ptr();
}

// Row stride of a matrix whose rows are dense but may lie apart. A single row's is its length: nobody
// steps by torch's stride of it, which may be anything (a sequence's length for its last position).
int64_t row_stride(const Tensor& t, const char* name) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "%s: the elements of a row must be adjacent%s", name);
  if (rows <= 1) return cols;
  if (t.stride(0) < cols) refuse(PyExc_ValueError, "%s: rows must not overlap%s", name);
  return t.stride(0);
}

int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large%s", name);
  return (int32_t)v;
}

// (a matrix whose rows row_stride has accepted, or a contiguous tensor)
Bytes bytes_of(const Tensor& t) {
  if (t.dim() != 2 || t.is_contiguous()) return dense_bytes(t.data_ptr(), (int64_t)t.nbytes());
  const int64_t e = (int64_t)t.element_size();
  return {(const char*)t.data_ptr(), t.numel() ? t.size(0) : 0, t.size(1) * e, t.stride(0) * e};
}
Bytes bytes_of(PyObject* o) { return o == Py_None ? Bytes{nullptr, 0, 0, 0} : bytes_of(THPVariable_Unpack(o)); }

// call(stream) with GPU `device` current, on torch's current stream of it.
template <class F>
int on_device(int device, F call) {
  const c10::hip::HIPStream stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device);
  c10::hip::OptionalHIPGuard guard;
  if (c10::hip::current_device() != device) guard.set_index((c10::DeviceIndex)device);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call((void*)stream.stream());
  Py_END_ALLOW_THREADS
  return rc;
}

// Runs f and turns C++ exceptions into Python's.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// route(logits, topk, scoring, bias, n_groups, topk_groups, group_score, renormalize, scale,
//       token_mask, topk_ids, topk_w, token_flags) -> (topk_ids, topk_w)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) refuse(PyExc_TypeError, "%s takes 13 arguments%s", "route");
    const Tensor& logits = *tensor_of(a[0], "logits");
    if (logits.dim() != 2) refuse(PyExc_ValueError, "%s must be a [T][E] tensor%s", "logits");
    const int64_t T = logits.size(0), E = logits.size(1);
    const int dev = logits.is_cuda() ? logits.get_device() : -1;
    check(logits, "logits", at::kFloat, {T, E}, dev);
    auto integer = [&](int i) {
      const long v = PyLong_AsLong(a[i]);
      if (v == -1 && PyErr_Occurred()) throw Refused{};
      if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large%s", "an argument");
      return (int32_t)v;
    };
    moe_lora_router r;
    r.T = size32(T, "T");
    r.n_experts = size32(E, "E");
    r.topk = integer(1);
    r.scoring = integer(2);
    r.n_groups = integer(4);
    r.topk_groups = integer(5);
    r.group_score = integer(6);
    r.renormalize = integer(7);
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
    r.scale = (float)scale;
    r.logits_stride = row_stride(logits, "logits");
    // (a topk that moe_lora_route refuses allocates nothing first)
    const int64_t k = r.topk > 0 && r.topk <= E ? r.topk : 0;
    Tensor ids, w;
    if (a[10] == Py_None) ids = at::empty({T, k}, logits.options().dtype(at::kInt));
    else ids = *tensor_of(a[10], "topk_ids");
    if (a[11] == Py_None) w = at::empty({T, k}, logits.options());
    else w = *tensor_of(a[11], "topk_w");
    check(ids, "topk_ids", at::kInt, {T, k}, dev);
    check(w, "topk_w", at::kFloat, {T, k}, dev);
    if (!ids.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "topk_ids");
    if (!w.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "topk_w");
    const void* bias = dense(a[3], "bias", at::kFloat, {E}, dev);
    const void* mask = dense(a[9], "token_mask", at::kBool, {T}, dev);
    void* flags = dense(a[12], "token_flags", at::kInt, {T}, dev);
    for (const int out : {10, 11, 12}) {
      if (a[out] == Py_None) continue;
      for (const int other : {0, 3, 9, 10, 11, 12})
        if (other != out && overlap(bytes_of(a[out]), bytes_of(a[other])))
          refuse(PyExc_ValueError, "%s overlaps another argument%s",
                 out == 10 ? "topk_ids" : out == 11 ? "topk_w" : "token_flags");
    }
    const int rc = on_device(dev, [&](void* stream) {
      return moe_lora_route((const float*)logits.data_ptr(), (const float*)bias, (const uint8_t*)mask, &r,
                            (int32_t*)ids.data_ptr(), (float*)w.data_ptr(), (int32_t*)flags, stream);
    });
    if (rc != MOELORA_OK) return PyLong_FromLong(rc);
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(ids)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(w)));
    return out;
  });
}

// linear(x, W, w_scale, bias, act, residual, y, workspace) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) refuse(PyExc_TypeError, "%s takes 8 arguments%s", "linear");
    const Tensor &x = *tensor_of(a[0], "x"), &W = *tensor_of(a[1], "W");
    if (x.dim() != 2 || W.dim() != 2) refuse(PyExc_ValueError, "%s must be [T][K] and W [N][K]%s", "x");
    const int64_t T = x.size(0), K = x.size(1), rows = W.size(0);
    const int dev = x.is_cuda() ? x.get_device() : -1;
    const bool w8 = a[2] != Py_None;
    moe_lora_linear_dims d;
    d.act = (int32_t)PyLong_AsLong(a[4]);
    if (d.act == -1 && PyErr_Occurred()) throw Refused{};
    const bool gated = d.act == MOELORA_ACT_SWIGLU;
    if (gated && rows % 2) refuse(PyExc_ValueError, "%s of swiglu has gate and up rows: an even number%s", "W");
    const int64_t N = gated ? rows / 2 : rows;
    check(x, "x", at::kBFloat16, {T, K}, dev);
    check(W, "W", w8 ? at::kByte : at::kBFloat16, {rows, K}, dev);
    const void* scale = dense(a[2], "w_scale", at::kFloat, {rows}, dev);
    const void* bias = dense(a[3], "bias", at::kBFloat16, {rows}, dev);
    d.T = size32(T, "T");
    d.in_features = size32(K, "K");
    d.out_features = size32(N, "N");
    d.w_type = w8 ? MOELORA_W_E4M3 : MOELORA_W_BF16;
    d.x_stride = row_stride(x, "x");
    d.w_stride = row_stride(W, "W");
    d.residual_stride = 0;
    const void* residual = nullptr;
    if (a[5] != Py_None) {
      const Tensor& r = *tensor_of(a[5], "residual");
      check(r, "residual", at::kBFloat16, {T, N}, dev);
      d.residual_stride = row_stride(r, "residual");
      residual = r.data_ptr();
    }
    Tensor y;
    if (a[6] == Py_None) {
      y = at::empty({T, N}, x.options());
    } else {
      y = *tensor_of(a[6], "y");
      check(y, "y", at::kBFloat16, {T, N}, dev);
    }
    d.y_stride = row_stride(y, "y");
    if (a[6] != Py_None) {
      const Bytes out = bytes_of(y);
      const bool in_place = residual == y.data_ptr() && (T == 1 || d.residual_stride == d.y_stride);
      for (const int i : {0, 1, 2, 3, 5})
        if (overlap(out, bytes_of(a[i])) && !(i == 5 && in_place))
          refuse(PyExc_ValueError, "%s overlaps an input%s", "y");
    }
    Tensor ws;
    if (a[7] != Py_None) {
      ws = *tensor_of(a[7], "workspace");
      check(ws, "workspace", at::kByte, ws.sizes(), dev);
      if (!ws.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "workspace");
      const size_t need = moe_lora_linear_workspace_size(&d);
      const Bytes used = dense_bytes(ws.data_ptr(), std::min((int64_t)need, ws.numel()));
      bool shares = overlap(used, bytes_of(y));
      for (const int i : {0, 1, 2, 3, 5}) shares |= overlap(used, bytes_of(a[i]));
      if (shares) refuse(PyExc_ValueError, "%s overlaps another argument%s", "workspace");
    } else if (const size_t need = moe_lora_linear_workspace_size(&d)) {
      ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
    }
    const int rc = on_device(dev, [&](void* stream) {
      return moe_lora_linear(x.data_ptr(), W.data_ptr(), (const float*)scale, bias, residual, &d, y.data_ptr(),
                             ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, stream);
    });
    if (rc != MOELORA_OK) return PyLong_FromLong(rc);
    if (a[6] != Py_None) return Py_NewRef(a[6]);
    return THPVariable_Wrap(std::move(y));
  });
}

PyMethodDef methods[] = {{"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, nullptr},
                         {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return nullptr;
  out_of_memory = PyObject_GetAttrString(torch, "OutOfMemoryError");
  Py_DECREF(torch);
  return out_of_memory ? PyModule_Create(&module) : nullptr;
}
