// Compiled half of the Python binding for the operators whose kernels take a few microseconds
// (moe_lora_route, moe_lora_linear, moe_lora_linear_lora, moe_lora_block_norm, moe_lora_forward_few):
// checks of torch tensors, outputs and workspaces from torch's allocator, torch's current stream, one call
// of the C ABI. As attribute reads and ctypes conversions in Python the same took 6 us of a 10 us call;
// here 1 us.
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
// linear_lora(.., A, B, adapter_ids) -> y
template <bool LORA>
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != (LORA ? 11 : 8)) refuse(PyExc_TypeError, "%s takes another number of arguments%s", "linear");
    const Tensor &x = *tensor_of(a[0], "x"), &W = *tensor_of(a[1], "W");
    if (x.dim() != 2 || W.dim() != 2) refuse(PyExc_ValueError, "%s must be [T][K] and W [N][K]%s", "x");
    const int64_t T = x.size(0), K = x.size(1), rows = W.size(0);
    const int dev = x.is_cuda() ? x.get_device() : -1;
    const bool w8 = a[2] != Py_None;
    moe_lora_linear_lora_dims dims;
    moe_lora_linear_dims& d = dims.linear;
    d.act = (int32_t)PyLong_AsLong(a[4]);
    if (d.act == -1 && PyErr_Occurred()) throw Refused{};
    const bool gated = d.act == MOELORA_ACT_SWIGLU;
    if (gated && rows % 2) refuse(PyExc_ValueError, "%s of swiglu has gate and up rows: an even number%s", "W");
    const int64_t N = gated ? rows / 2 : rows;
    check(x, "x", at::kBFloat16, {T, K}, dev);
    check(W, "W", w8 ? at::kByte : at::kBFloat16, {rows, K}, dev);
    const void* scale = dense(a[2], "w_scale", at::kFloat, {rows}, dev);
    const void* bias = dense(a[3], "bias", at::kBFloat16, {rows}, dev);
    const void *A = nullptr, *B = nullptr, *ids = nullptr;
    if (LORA) {
      const Tensor& ta = *tensor_of(a[8], "A");
      if (ta.dim() != 3) refuse(PyExc_ValueError, "%s must be [n_adapters][rank][K]%s", "A");
      const int64_t nA = ta.size(0), r = ta.size(1);
      A = dense(a[8], "A", at::kBFloat16, {nA, r, K}, dev);
      tensor_of(a[9], "B");
      B = dense(a[9], "B", at::kBFloat16, {nA, rows, r}, dev);
      tensor_of(a[10], "adapter_ids");
      ids = dense(a[10], "adapter_ids", at::kInt, {T}, dev);
      dims.n_adapters = size32(nA, "n_adapters");
      dims.rank = size32(r, "rank");
    }
    const auto workspace_size = [&] {
      return LORA ? moe_lora_linear_lora_workspace_size(&dims) : moe_lora_linear_workspace_size(&d);
    };
    constexpr int inputs[] = {0, 1, 2, 3, 5, 8, 9, 10};
    constexpr int n_inputs = LORA ? 8 : 5;
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
      for (int j = 0; j < n_inputs; ++j) {
        const int i = inputs[j];
        if (overlap(out, bytes_of(a[i])) && !(i == 5 && in_place))
          refuse(PyExc_ValueError, "%s overlaps an input%s", "y");
      }
    }
    Tensor ws;
    if (a[7] != Py_None) {
      ws = *tensor_of(a[7], "workspace");
      check(ws, "workspace", at::kByte, ws.sizes(), dev);
      if (!ws.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "workspace");
      const size_t need = workspace_size();
      const Bytes used = dense_bytes(ws.data_ptr(), std::min((int64_t)need, ws.numel()));
      bool shares = overlap(used, bytes_of(y));
      for (int j = 0; j < n_inputs; ++j) shares |= overlap(used, bytes_of(a[inputs[j]]));
      if (shares) refuse(PyExc_ValueError, "%s overlaps another argument%s", "workspace");
    } else if (const size_t need = workspace_size()) {
      ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
    }
    const int rc = on_device(dev, [&](void* stream) {
      void* const at = ws.defined() ? ws.data_ptr() : nullptr;
      const size_t bytes = ws.defined() ? (size_t)ws.numel() : 0;
      if (LORA)
        return moe_lora_linear_lora(x.data_ptr(), W.data_ptr(), (const float*)scale, bias, residual, A, B,
                                    (const int32_t*)ids, &dims, y.data_ptr(), at, bytes, stream);
      return moe_lora_linear(x.data_ptr(), W.data_ptr(), (const float*)scale, bias, residual, &d, y.data_ptr(),
                             at, bytes, stream);
    });
    if (rc != MOELORA_OK) return PyLong_FromLong(rc);
    if (a[6] != Py_None) return Py_NewRef(a[6]);
    return THPVariable_Wrap(std::move(y));
  });
}

// block_norm(y, residual, gate, sigmoid, post_weight, post_bias, weight, bias, norm, eps, residual_scale,
//            branch_scale, sum, out) -> (sum, out)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14) refuse(PyExc_TypeError, "%s takes 14 arguments%s", "block_norm");
    const Tensor& res = *tensor_of(a[1], "residual");
    if (res.dim() != 2) refuse(PyExc_ValueError, "%s must be a [T][h] tensor%s", "residual");
    const int64_t T = res.size(0), h = res.size(1);
    const int dev = res.is_cuda() ? res.get_device() : -1;
    moe_lora_block_norm_dims d = {};
    d.T = size32(T, "T");
    d.hidden = size32(h, "h");
    auto matrix = [&](PyObject* o, const char* name, int64_t* stride) -> void* {
      if (o == Py_None) return nullptr;
      const Tensor& t = *tensor_of(o, name);
      check(t, name, at::kBFloat16, {T, h}, dev);
      *stride = row_stride(t, name);
      return t.data_ptr();
    };
    auto number = [&](int i) {
      const double v = PyFloat_AsDouble(a[i]);
      if (v == -1.0 && PyErr_Occurred()) throw Refused{};
      return (float)v;
    };
    const void* residual = matrix(a[1], "residual", &d.residual_stride);
    const void* y = matrix(a[0], "y", &d.y_stride);
    const void* gate = nullptr;
    Bytes gate_bytes = {nullptr, 0, 0, 0};
    d.gate = MOELORA_GATE_NONE;
    if (a[2] != Py_None) {
      const Tensor& g = *tensor_of(a[2], "gate");
      const long sigmoid = PyLong_AsLong(a[3]);
      if (sigmoid == -1 && PyErr_Occurred()) throw Refused{};
      if (g.dim() == 1) {
        gate = dense(a[2], "gate", at::kFloat, {T}, dev);
        d.gate = sigmoid ? MOELORA_GATE_SIGMOID : MOELORA_GATE_TOKEN;
        gate_bytes = bytes_of(g);
      } else {
        check(g, "gate", at::kBFloat16, {T, h}, dev);
        if (sigmoid) refuse(PyExc_ValueError, "%s: the sigmoid is of a [T] gate%s", "sigmoid_gate");
        if (T > 1 && g.stride(0) == 0) {  // one row for every token
          if (h > 1 && g.stride(1) != 1) refuse(PyExc_ValueError, "%s: the elements of a row must be adjacent%s", "gate");
          gate_bytes = dense_bytes(g.data_ptr(), 2 * h);
        } else {
          d.gate_stride = row_stride(g, "gate");
          gate_bytes = bytes_of(g);
        }
        gate = g.data_ptr();
        d.gate = MOELORA_GATE_FEATURES;
      }
    }
    const void* vectors[4];
    const char* const names[] = {"post_weight", "post_bias", "weight", "bias"};
    for (int i = 0; i < 4; ++i) vectors[i] = dense(a[4 + i], names[i], at::kBFloat16, {h}, dev);
    const long norm = PyLong_AsLong(a[8]);
    if (norm == -1 && PyErr_Occurred()) throw Refused{};
    d.norm = (int32_t)norm;
    d.eps = number(9);
    d.residual_scale = number(10);
    d.branch_scale = number(11);
    Tensor sum, out;
    if (a[12] != Py_None) sum = *tensor_of(a[12], "total");
    else if (a[0] != Py_None) sum = at::empty({T, h}, res.options());
    if (a[13] != Py_None) out = *tensor_of(a[13], "out");
    else if (a[6] != Py_None) out = at::empty({T, h}, res.options());
    for (const Tensor* t : {&sum, &out}) {
      if (!t->defined()) continue;
      const char* name = t == &sum ? "total" : "out";
      check(*t, name, at::kBFloat16, {T, h}, dev);
      int64_t& stride = t == &sum ? d.sum_stride : d.out_stride;
      stride = row_stride(*t, name);
      if (a[t == &sum ? 12 : 13] == Py_None) continue;
      const Bytes b = bytes_of(*t);
      bool shares = overlap(b, gate_bytes);
      for (int i = 4; i < 8; ++i) shares |= overlap(b, bytes_of(a[i]));
      for (int i = 0; i < 2; ++i) {
        const bool same = a[i] != Py_None && THPVariable_Unpack(a[i]).data_ptr() == t->data_ptr() &&
                          (T == 1 || (i ? d.residual_stride : d.y_stride) == stride);
        shares |= overlap(b, bytes_of(a[i])) && !same;
      }
      const Tensor& other = t == &sum ? out : sum;
      shares |= other.defined() && overlap(b, bytes_of(other));
      if (shares) refuse(PyExc_ValueError, "%s overlaps another argument%s", name);
    }
    const int rc = on_device(dev, [&](void* stream) {
      return moe_lora_block_norm(y, residual, gate, vectors[0], vectors[1], vectors[2], vectors[3], &d,
                                 sum.defined() ? sum.data_ptr() : nullptr, out.defined() ? out.data_ptr() : nullptr,
                                 stream);
    });
    if (rc != MOELORA_OK) return PyLong_FromLong(rc);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    for (int i = 0; i < 2; ++i) {
      Tensor& t = i ? out : sum;
      PyTuple_SET_ITEM(pair, i, t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None));
    }
    return pair;
  });
}

// forward_few(x, W1, W2, A1, B1, A2, B2, adapter_ids, router_logits, topk, topk_ids, topk_w, W1_scale,
//             W2_scale, y, workspace) -> y
PyObject* forward_few(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 16) refuse(PyExc_TypeError, "%s takes 16 arguments%s", "forward_few");
    const Tensor &x = *tensor_of(a[0], "x"), &W1 = *tensor_of(a[1], "W1"), &A1 = *tensor_of(a[3], "A1");
    if (x.dim() != 2 || W1.dim() != 3 || A1.dim() != 4)
      refuse(PyExc_ValueError, "%s must be [T][h], W1 [E][2I][h] and A1 [n_adapters][E][rank][h]%s", "x");
    const int64_t T = x.size(0), h = x.size(1), E = W1.size(0), I = W1.size(1) / 2, nA = A1.size(0), r = A1.size(2);
    const int dev = x.is_cuda() ? x.get_device() : -1;
    const bool w8 = a[12] != Py_None;
    if (w8 != (a[13] != Py_None)) refuse(PyExc_ValueError, "%s and W2_scale go together%s", "W1_scale");
    const at::ScalarType wt = w8 ? at::kByte : at::kBFloat16;
    for (int i = 0; i < 8; ++i) tensor_of(a[i], "each of x, W1, W2, A1, B1, A2, B2 and adapter_ids");
    const void* px = dense(a[0], "x", at::kBFloat16, {T, h}, dev);
    const void* pW1 = dense(a[1], "W1", wt, {E, 2 * I, h}, dev);
    const void* pW2 = dense(a[2], "W2", wt, {E, h, I}, dev);
    const void* pA1 = dense(a[3], "A1", at::kBFloat16, {nA, E, r, h}, dev);
    const void* pB1 = dense(a[4], "B1", at::kBFloat16, {nA, E, 2 * I, r}, dev);
    const void* pA2 = dense(a[5], "A2", at::kBFloat16, {nA, E, r, I}, dev);
    const void* pB2 = dense(a[6], "B2", at::kBFloat16, {nA, E, h, r}, dev);
    const void* pids = dense(a[7], "adapter_ids", at::kInt, {T}, dev);
    const void* ps1 = dense(a[12], "W1_scale", at::kFloat, {E, 2 * I}, dev);
    const void* ps2 = dense(a[13], "W2_scale", at::kFloat, {E, h}, dev);
    const bool routes = a[8] != Py_None;
    if (routes == (a[10] != Py_None) || (a[10] != Py_None) != (a[11] != Py_None))
      refuse(PyExc_ValueError, "either %s and topk, or topk_ids and topk_w%s", "router_logits");
    int64_t k;
    if (routes) {
      k = PyLong_AsLong(a[9]);
      if (k == -1 && PyErr_Occurred()) throw Refused{};
    } else {
      const Tensor& ids = *tensor_of(a[10], "topk_ids");
      if (ids.dim() != 2) refuse(PyExc_ValueError, "%s must be a [T][k] tensor%s", "topk_ids");
      k = ids.size(1);
      if (a[9] != Py_None) {
        const long given = PyLong_AsLong(a[9]);
        if (given == -1 && PyErr_Occurred()) throw Refused{};
        if (given != k) refuse(PyExc_ValueError, "%s is not the number of topk_ids' columns%s", "topk");
      }
    }
    if (k < INT32_MIN || k > INT32_MAX) refuse(PyExc_ValueError, "%s is too large%s", "topk");
    const void* logits = dense(a[8], "router_logits", at::kFloat, {T, E}, dev);
    const void* tids = dense(a[10], "topk_ids", at::kInt, {T, k}, dev);
    const void* tw = dense(a[11], "topk_w", at::kFloat, {T, k}, dev);
    moe_lora_dims d;
    d.T = size32(T, "T");
    d.hidden = size32(h, "h");
    d.inter = size32(I, "I");
    d.n_experts = size32(E, "E");
    d.n_adapters = size32(nA, "n_adapters");
    d.rank = size32(r, "rank");
    const size_t need = moe_lora_few_workspace_size(&d, (int32_t)k);
    if (!need) return PyLong_FromLong(MOELORA_EINVAL_DIMS);
    constexpr int inputs[] = {0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 12, 13};
    Tensor y, ws;
    if (a[14] == Py_None) {
      y = at::empty({T, h}, x.options());
    } else {
      dense(a[14], "y", at::kBFloat16, {T, h}, dev);
      y = *tensor_of(a[14], "y");
      for (const int i : inputs)
        if (overlap(bytes_of(y), bytes_of(a[i]))) refuse(PyExc_ValueError, "%s overlaps an input%s", "y");
    }
    if (a[15] == Py_None) {
      ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
    } else {
      ws = *tensor_of(a[15], "workspace");
      check(ws, "workspace", at::kByte, ws.sizes(), dev);
      if (!ws.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "workspace");
      const Bytes used = dense_bytes(ws.data_ptr(), std::min((int64_t)need, ws.numel()));
      bool shares = overlap(used, bytes_of(y));
      for (const int i : inputs) shares |= overlap(used, bytes_of(a[i]));
      if (shares) refuse(PyExc_ValueError, "%s overlaps another argument%s", "workspace");
    }
    const int rc = on_device(dev, [&](void* stream) {
      return moe_lora_forward_few(px, (const float*)logits, (const int32_t*)tids, (const float*)tw, pW1,
                                  (const float*)ps1, pW2, (const float*)ps2, pA1, pB1, pA2, pB2,
                                  (const int32_t*)pids, (int32_t)k, &d, y.data_ptr(), ws.data_ptr(),
                                  (size_t)ws.numel(), stream);
    });
    if (rc != MOELORA_OK) return PyLong_FromLong(rc);
    if (a[14] != Py_None) return Py_NewRef(a[14]);
    return THPVariable_Wrap(std::move(y));
  });
}

PyMethodDef methods[] = {{"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, nullptr},
                         {"linear", (PyCFunction)(void (*)(void))linear<false>, METH_FASTCALL, nullptr},
                         {"linear_lora", (PyCFunction)(void (*)(void))linear<true>, METH_FASTCALL, nullptr},
                         {"block_norm", (PyCFunction)(void (*)(void))block_norm, METH_FASTCALL, nullptr},
                         {"forward_few", (PyCFunction)(void (*)(void))forward_few, METH_FASTCALL, nullptr},
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
