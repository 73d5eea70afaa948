// Native calls of the MoE block's binding (block.py), for the common case: operands of the right types
// and shapes (rows may have a stride), outputs to be allocated, the current stream. Each function checks that
// case, allocates, and calls the C entry point whose address it is given; it returns None for
// anything else, also where the entry point refuses, and the Python function then takes its own path
// and raises what there is to raise. A call costs a third of the Python path's host time, which is
// what the smallest calls take outside a CUDA graph.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "mol_block.h"

namespace {

using at::Tensor;

// A tensor on the current device, which is the one that a call launches on; asked for once a call.
thread_local int current = -1;
bool here(const Tensor& t) {
  if (!t.is_cuda()) return false;
  if (current < 0) current = c10::cuda::current_device();
  return t.get_device() == current;
}

// A plain tensor on the GPU, contiguous, of the type and shape; sizes of -1 match any.
bool fits(const Tensor& t, at::ScalarType type, c10::IntArrayRef sizes) {
  if (t.scalar_type() != type || !here(t) || t.dim() != (int64_t)sizes.size() ||
      !t.is_contiguous())
    return false;
  for (size_t i = 0; i < sizes.size(); ++i)
    if (sizes[i] >= 0 && t.sizes()[i] != sizes[i]) return false;
  return true;
}

// A plain tensor of rows on the GPU, its columns neighbours; the row stride of a single row (or none)
// does not matter.
bool rows_fit(const Tensor& t, at::ScalarType type, int64_t rows, int64_t columns, int64_t& stride) {
  if (t.scalar_type() != type || !here(t) || t.dim() != 2 || t.size(0) != rows ||
      t.size(1) != columns || (t.stride(1) != 1 && columns > 1))
    return false;
  stride = rows > 1 ? t.stride(0) : (columns + 7) / 8 * 8;
  return true;
}

const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// Arguments in their order: each take_* returns false when the argument is not of its kind.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  bool take(void*& p) {
    if (i >= n || !PyLong_CheckExact(v[i])) return false;
    p = PyLong_AsVoidPtr(v[i++]);
    return p != nullptr;
  }
  bool take(const Tensor*& t) { return i < n && (t = tensor(v[i++])); }
  bool take_optional(const Tensor*& t) {
    t = nullptr;
    if (i >= n) return false;
    PyObject* o = v[i++];
    return o == Py_None || (t = tensor(o));
  }
  bool take(int64_t& x) {
    if (i >= n || !PyLong_CheckExact(v[i])) return false;
    x = PyLong_AsLongLong(v[i++]);
    return !PyErr_Occurred();
  }
  bool take(double& x) {
    if (i >= n) return false;
    x = PyFloat_AsDouble(v[i++]);
    return !PyErr_Occurred();
  }
};

// Weight rows [lead..., K] as the Python side hands them over: data, scales or None, inputs, group.
struct Weights {
  const Tensor *data, *scales;
  int64_t K, group;
  bool take(Args& a) {
    return a.take(data) && a.take_optional(scales) && a.take(K) && a.take(group) &&
           data->dim() >= 1;
  }
  bool fits_rows(int64_t lead, int64_t N) const {
    if (!scales) return group == 0 && fits(*data, at::kBFloat16, {lead, N, K});
    if (group != 32 && group != 64 && group != 128) return false;
    const int64_t Kp = (K + 255) / 256 * 256;
    return fits(*data, at::kByte, {lead, N, Kp / 2}) && fits(*scales, at::kBFloat16, {lead, N, Kp / group});
  }
  const void* scale_ptr() const { return scales ? scales->data_ptr() : nullptr; }
};

void* stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* pair(const Tensor& a, PyObject* second) {
  PyObject* first = THPVariable_Wrap(a);
  PyObject* out = first && second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return out;
}

// C++ exceptions (an allocation that fails) become the Python path's to meet again.
template <PyObject* (*F)(Args)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  current = -1;
  try {
    return F(Args{args, n});
  } catch (const std::exception&) {
    return none();
  }
}

bool small(std::initializer_list<int64_t> sizes) {
  for (int64_t s : sizes)
    if (s < 0 || s > INT32_MAX) return false;
  return true;
}

PyObject* block_norm(Args a) {
  void* f;
  const Tensor *y, *residual, *pre, *post, *gate;
  double scale, eps;
  if (!a.take(f) || !a.take(y) || !a.take(residual) || !a.take_optional(pre) ||
      !a.take_optional(post) || !a.take_optional(gate) || !a.take(scale) || !a.take(eps))
    return none();
  if (y->dim() != 2) return none();
  const int64_t T = y->size(0), H = y->size(1);
  int64_t ys, rs, gs = 0;
  if (!small({T, H}) || !rows_fit(*y, at::kBFloat16, T, H, ys) ||
      !rows_fit(*residual, at::kBFloat16, T, H, rs) || (pre && !fits(*pre, at::kBFloat16, {H})) ||
      (post && !fits(*post, at::kBFloat16, {H})))
    return none();
  if (gate && !(gate->dim() == 2 ? rows_fit(*gate, at::kBFloat16, T, H, gs)
                                 : fits(*gate, at::kBFloat16, {H})))
    return none();
  Tensor out = at::empty({T, H}, y->options()), normed;
  if (pre) normed = at::empty({T, H}, y->options());
  auto ptr = [](const Tensor* t) -> const void* { return t ? t->data_ptr() : nullptr; };
  const int32_t status = reinterpret_cast<decltype(&mol_block_norm)>(f)(
      y->data_ptr(), ys, residual->data_ptr(), rs, ptr(post), ptr(gate), gs,
      (float)scale, ptr(pre), (float)eps, T, (int32_t)H, out.data_ptr(), H,
      pre ? normed.data_ptr() : nullptr, pre ? H : 0, stream_of(*y));
  if (status != MOL_OK) return none();
  return pair(out, pre ? THPVariable_Wrap(normed) : Py_NewRef(Py_None));
}

PyObject* moe_route(Args a) {
  void* f;
  const Tensor* logits;
  int64_t topk, renormalize;
  double scale;
  if (!a.take(f) || !a.take(logits) || !a.take(topk) || !a.take(renormalize) || !a.take(scale))
    return none();
  const bool bf16 = logits->scalar_type() == at::kBFloat16;
  if (logits->dim() != 2) return none();
  const int64_t T = logits->size(0), E = logits->size(1);
  int64_t stride;
  if (!small({T, E, topk}) ||
      !rows_fit(*logits, bf16 ? at::kBFloat16 : at::kFloat, T, E, stride))
    return none();
  Tensor ids = at::empty({T, topk}, logits->options().dtype(at::kInt));
  Tensor weights = at::empty({T, topk}, logits->options().dtype(at::kFloat));
  const int32_t status = reinterpret_cast<decltype(&mol_moe_route)>(f)(
      logits->data_ptr(), bf16 ? MOL_BF16 : MOL_F32, stride, T, (int32_t)E, (int32_t)topk,
      (int32_t)renormalize, (float)scale, static_cast<int32_t*>(ids.data_ptr()),
      static_cast<float*>(weights.data_ptr()), stream_of(*logits));
  return status == MOL_OK ? pair(ids, THPVariable_Wrap(weights)) : none();
}

PyObject* moe_gate_up(Args a) {
  void* f;
  const Tensor *x, *ids, *delta;
  Weights w;
  if (!a.take(f) || !a.take(x) || !a.take(ids) || !w.take(a) || !a.take_optional(delta) ||
      w.data->dim() != 3)
    return none();
  const int64_t E = w.data->size(0), I2 = w.data->size(1);
  if (x->dim() != 2 || !w.fits_rows(E, I2)) return none();
  const int64_t T = x->size(0), H = w.K;
  int64_t xs, ds = 0;
  if (!fits(*ids, at::kInt, {T, -1}) || !rows_fit(*x, at::kBFloat16, T, H, xs)) return none();
  const int64_t k = ids->size(1);
  if (!small({T, k, E, H, I2}) || I2 % 2 ||
      (delta && !rows_fit(*delta, at::kBFloat16, T * k, I2, ds)))
    return none();
  Tensor act = at::empty({T * k, I2 / 2}, x->options());
  const int32_t status = reinterpret_cast<decltype(&mol_moe_gate_up)>(f)(
      x->data_ptr(), xs, static_cast<const int32_t*>(ids->data_ptr()), T, (int32_t)k, (int32_t)E,
      (int32_t)H, (int32_t)(I2 / 2), w.data->data_ptr(), w.scale_ptr(), (int32_t)w.group,
      delta ? delta->data_ptr() : nullptr, ds, act.data_ptr(), stream_of(*x));
  return status == MOL_OK ? THPVariable_Wrap(act) : none();
}

Tensor scratch(const Tensor& like, size_t bytes) {
  return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : Tensor();
}

PyObject* moe_down(Args a) {
  void *f, *need;
  const Tensor *act, *ids, *weights, *delta;
  Weights w;
  if (!a.take(f) || !a.take(need) || !a.take(act) || !a.take(ids) || !a.take(weights) ||
      !w.take(a) || !a.take_optional(delta) || w.data->dim() != 3)
    return none();
  const int64_t E = w.data->size(0), H = w.data->size(1), I = w.K;
  if (!fits(*ids, at::kInt, {-1, -1}) || !w.fits_rows(E, H)) return none();
  const int64_t T = ids->size(0), k = ids->size(1);
  int64_t ds = 0;
  if (!small({T, k, E, H, I}) || !fits(*act, at::kBFloat16, {T * k, I}) ||
      !fits(*weights, at::kFloat, {T, k}) ||
      (delta && !rows_fit(*delta, at::kBFloat16, T * k, H, ds)))
    return none();
  const size_t bytes = reinterpret_cast<decltype(&mol_moe_workspace_bytes)>(need)(
      T, (int32_t)k, (int32_t)E, (int32_t)H, (int32_t)I, (int32_t)w.group);
  Tensor out = at::empty({T, H}, act->options()), ws = scratch(*act, bytes);
  const int32_t status = reinterpret_cast<decltype(&mol_moe_down_split)>(f)(
      act->data_ptr(), static_cast<const int32_t*>(ids->data_ptr()),
      static_cast<const float*>(weights->data_ptr()), T, (int32_t)k, (int32_t)E, (int32_t)H,
      (int32_t)I, w.data->data_ptr(), w.scale_ptr(), (int32_t)w.group,
      delta ? delta->data_ptr() : nullptr, ds, bytes ? ws.data_ptr() : nullptr, bytes,
      out.data_ptr(), H, stream_of(*act));
  return status == MOL_OK ? THPVariable_Wrap(out) : none();
}

PyObject* moe_forward(Args a) {
  void *f, *need;
  const Tensor *x, *ids, *weights;
  Weights gu, dn;
  if (!a.take(f) || !a.take(need) || !a.take(x) || !a.take(ids) || !a.take(weights) ||
      !gu.take(a) || !dn.take(a) || gu.data->dim() != 3 || dn.data->dim() != 3)
    return none();
  const int64_t E = gu.data->size(0), I = dn.K, H = gu.K;
  if (gu.group != dn.group || x->dim() != 2 || !gu.fits_rows(E, 2 * I) || !dn.fits_rows(E, H))
    return none();
  const int64_t T = x->size(0);
  int64_t xs;
  if (!fits(*ids, at::kInt, {T, -1}) || !rows_fit(*x, at::kBFloat16, T, H, xs)) return none();
  const int64_t k = ids->size(1);
  if (!small({T, k, E, H, I}) || !fits(*weights, at::kFloat, {T, k})) return none();
  const size_t bytes = reinterpret_cast<decltype(&mol_moe_workspace_bytes)>(need)(
      T, (int32_t)k, (int32_t)E, (int32_t)H, (int32_t)I, (int32_t)gu.group);
  Tensor out = at::empty({T, H}, x->options()), act = at::empty({T * k, I}, x->options());
  Tensor ws = scratch(*x, bytes);
  const int32_t status = reinterpret_cast<decltype(&mol_moe_forward_split)>(f)(
      x->data_ptr(), xs, static_cast<const int32_t*>(ids->data_ptr()),
      static_cast<const float*>(weights->data_ptr()), T, (int32_t)k, (int32_t)E, (int32_t)H,
      (int32_t)I, gu.data->data_ptr(), gu.scale_ptr(), dn.data->data_ptr(), dn.scale_ptr(),
      (int32_t)gu.group, act.data_ptr(), bytes ? ws.data_ptr() : nullptr, bytes, out.data_ptr(), H,
      stream_of(*x));
  return status == MOL_OK ? THPVariable_Wrap(out) : none();
}

PyObject* w4_linear(Args a) {
  void* f;
  const Tensor* x;
  Weights w;
  if (!a.take(f) || !a.take(x) || !w.take(a) || w.data->dim() != 2 || !w.scales) return none();
  const int64_t N = w.data->size(0), K = w.K;
  if (x->dim() != 2 || (w.group != 32 && w.group != 64 && w.group != 128))
    return none();
  const int64_t T = x->size(0), Kp = (K + 255) / 256 * 256;
  int64_t xs;
  if (!small({T, N, K}) || !rows_fit(*x, at::kBFloat16, T, K, xs) || !fits(*w.data, at::kByte, {N, Kp / 2}) ||
      !fits(*w.scales, at::kBFloat16, {N, Kp / w.group}))
    return none();
  Tensor out = at::empty({T, N}, x->options());
  const int32_t status = reinterpret_cast<decltype(&mol_w4_linear)>(f)(
      x->data_ptr(), xs, T, (int32_t)K, (int32_t)N, w.data->data_ptr(), w.scale_ptr(),
      (int32_t)w.group, out.data_ptr(), N, stream_of(*x));
  return status == MOL_OK ? THPVariable_Wrap(out) : none();
}

#define MOL_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOL_METHOD(block_norm), MOL_METHOD(moe_route), MOL_METHOD(moe_gate_up),
                         MOL_METHOD(moe_down),   MOL_METHOD(moe_forward), MOL_METHOD(w4_linear),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_native() { return PyModule_Create(&module); }
