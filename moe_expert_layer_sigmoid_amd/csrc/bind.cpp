// The short way from a Python call of a linear operator to the C ABI.  The
// smallest of these calls take 2 to 5 us on the GPU, of which a launch needs
// 2.5 us of host time; checking three tensors and reading their addresses from
// Python took as long again (5.6 us a call of the quantiser).
//
// Each function returns the status of the C call, or None if an argument is
// not what it expects: the caller then takes the checks in Python, which name
// the argument that is wrong.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

constexpr at::ScalarType kTypes[] = {at::kBFloat16, at::kHalf, at::kFloat, at::kFloat8_e4m3fn};  // moe_type_t

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// A device tensor.  (data_ptr() throws for a subclass without storage of its own;
// the caller then takes the checks in Python.)
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() ? &t : nullptr;
}

// The address of a contiguous tensor of the type, on the device, with at least n elements.
struct Args {
  int dev;
  bool ok = true;
  void* of(PyObject* o, at::ScalarType type, int64_t n) {
    const at::Tensor* t = ok ? tensor(o) : nullptr;
    if (!t || t->device().index() != dev || !t->is_contiguous() || t->numel() < n ||
        !(t->scalar_type() == type || (type == at::kFloat8_e4m3fn && t->scalar_type() == at::kByte))) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
};

// The stream of a call: None is the device's current one.
bool stream_of(PyObject* o, int dev, moe_stream_t* st) {
  if (dev != c10::hip::current_device()) return false;
  if (o != Py_None) return false;
  *st = reinterpret_cast<moe_stream_t>(c10::hip::getCurrentHIPStream(dev).stream());
  return true;
}

// quant(swiglu, x, q, qs, stream)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) Py_RETURN_NONE;
  try {
    const bool swiglu = a[0] == Py_True;
    const at::Tensor* x = tensor(a[1]);
    if (!x || x->dim() != 2) Py_RETURN_NONE;
    const int64_t parts = swiglu ? 2 : 1, rows = x->size(0), K = x->size(1) / parts;
    int type = 0;
    while (type < 3 && kTypes[type] != x->scalar_type()) ++type;
    const int64_t ldx = rows > 1 ? x->stride(0) : parts * K;
    if (type == 3 || x->size(1) != parts * K || (x->numel() && x->stride(1) != 1) || ldx < parts * K ||
        rows > INT32_MAX || K > INT32_MAX)
      Py_RETURN_NONE;
    Args c{x->device().index()};
    auto* q = static_cast<uint8_t*>(c.of(a[2], at::kFloat8_e4m3fn, rows * K));
    auto* qs = static_cast<float*>(c.of(a[3], at::kFloat, rows * blocks(K)));
    moe_stream_t st;
    if (!c.ok || !stream_of(a[4], c.dev, &st)) Py_RETURN_NONE;
    return PyLong_FromLong((swiglu ? moe_fp8_swiglu_quant : moe_fp8_quant)(
        (int32_t)rows, (int32_t)K, type, x->data_ptr(), ldx, q, qs, st));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// The descriptor behind a ctypes structure.
bool descriptor(PyObject* o, moe_linear_t* d) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool ok = b.len == (Py_ssize_t)sizeof(*d);
  if (ok) memcpy(d, b.buf, sizeof(*d));
  PyBuffer_Release(&b);
  return ok && d->in_type >= 0 && d->in_type <= MOE_TYPE_FP8 && d->out_type >= 0 && d->out_type <= MOE_TYPE_FP8;
}

bool rest(Args& c, const moe_linear_t& d, PyObject* scratch, PyObject* offsets, void** ws, size_t* bytes,
          const int32_t** off) {
  *ws = nullptr;
  *bytes = 0;
  *off = nullptr;
  if (scratch != Py_None) {
    *ws = c.of(scratch, at::kByte, 0);
    if (c.ok) *bytes = (size_t)THPVariable_Unpack(scratch).numel();
  }
  if (offsets != Py_None) *off = static_cast<const int32_t*>(c.of(offsets, at::kInt, (int64_t)d.groups + 1));
  return c.ok;
}

// fp8(d, xq, xs, w, ws, y, scratch, offsets, stream)
PyObject* fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  moe_linear_t d;
  if (n != 9) Py_RETURN_NONE;
  try {
    const at::Tensor* y = tensor(a[5]);
    if (!y || !descriptor(a[0], &d)) Py_RETURN_NONE;
    Args c{y->device().index()};
    const int64_t R = d.rows, N = d.N, K = d.K, G = d.groups;
    auto* xq = static_cast<const uint8_t*>(c.of(a[1], at::kFloat8_e4m3fn, R * K));
    auto* xs = static_cast<const float*>(c.of(a[2], at::kFloat, R * blocks(K)));
    auto* w = static_cast<const uint8_t*>(c.of(a[3], at::kFloat8_e4m3fn, G * N * K));
    auto* ws = static_cast<const float*>(c.of(a[4], at::kFloat, G * blocks(N) * blocks(K)));
    void* out = c.of(a[5], kTypes[d.out_type], R * N);
    void* scratch;
    size_t bytes;
    const int32_t* off;
    moe_stream_t st;
    if (!rest(c, d, a[6], a[7], &scratch, &bytes, &off) || !stream_of(a[8], c.dev, &st)) Py_RETURN_NONE;
    return PyLong_FromLong(moe_fp8_linear(&d, xq, xs, w, ws, off, out, scratch, bytes, st));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// grouped(op, d, a, b, out, scratch, offsets, stream); op 0: x w -> y, 1: dy w -> dx, 2: dy x -> dw
PyObject* grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  moe_linear_t d;
  if (n != 8) Py_RETURN_NONE;
  try {
    const long op = PyLong_AsLong(a[0]);
    const at::Tensor* y = tensor(a[4]);
    if (op < 0 || op > 2 || !y || !descriptor(a[1], &d)) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    Args c{y->device().index()};
    const int64_t R = d.rows, x = R * d.K, dy = R * d.N, w = (int64_t)d.groups * d.N * d.K;
    const int64_t need[3][3] = {{x, w, dy}, {dy, w, x}, {dy, x, w}};
    const void* p = c.of(a[2], kTypes[d.in_type], need[op][0]);
    const void* q = c.of(a[3], kTypes[d.in_type], need[op][1]);
    void* out = c.of(a[4], kTypes[d.out_type], need[op][2]);
    void* scratch;
    size_t bytes;
    const int32_t* off;
    moe_stream_t st;
    if (!rest(c, d, a[5], a[6], &scratch, &bytes, &off) || !stream_of(a[7], c.dev, &st)) Py_RETURN_NONE;
    const auto f = op == 0 ? moe_grouped_linear : op == 1 ? moe_grouped_linear_dx : moe_grouped_linear_dw;
    return PyLong_FromLong(f(&d, p, q, off, out, scratch, bytes, st));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {{"quant", fast(quant), METH_FASTCALL, nullptr},
                          {"fp8", fast(fp8), METH_FASTCALL, nullptr},
                          {"grouped", fast(grouped), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers and libraries this was built against.
// Nothing here touches a tensor before the caller has compared it.
PyMODINIT_FUNC PyInit__bind() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "torch_version", MOE_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
