// The call of an entry point from Python without ctypes: a callable that takes the params structure
// and tensors, checks the tensors (on the current device, contiguous, of the types that the entry
// point reads and writes, and large enough) and calls the function with their addresses and the handle of the current stream, or of
// the one that is given behind them.
// Where anything is out of the ordinary (a raw pointer, a tensor that the kernel could not read)
// it calls nothing and returns None, and the binding in Python, which says what is wrong, goes on.
// Through ctypes and the tensors' methods a call of one row's norm takes 7.2 us with its launch, this
// way 3.1 us.  Tensors are looked at through DLPack's exchange interface.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>
#include <string.h>

#include "dsv4.h"

namespace {

constexpr int kMaxTensors = 8;

// What an argument holds: anything, the activations' type, the logits', floats and integers of 32
// bits, e4m3, the experts' rows (e4m3 with scales, else the activations' type).
enum Holds : unsigned { kAny, kAct, kLogits, kF32, kI32, kE4m3, kRows };

struct Entry {
  void* function;
  int tensors;      // arguments between the params and the stream
  unsigned holds;   // of the i-th: 4 bits from 4 i on
  int sized;        // 1: the bytes of the last one are an argument, behind it
};

const DLPackExchangeAPI* g_api = nullptr;
PyTypeObject* g_tensor = nullptr;  // torch.Tensor
PyObject* g_device = nullptr;      // () -> the current CUDA device

PyObject* attribute(PyObject* o, const char* name) {
  PyObject* v = o ? PyObject_GetAttrString(o, name) : nullptr;
  PyErr_Clear();
  return v;
}

// What the calls need of torch, once it has been imported; it lives as long as the interpreter.
bool find_torch() {
  if (g_api) return true;
  PyObject* torch = PyDict_GetItemString(PyImport_GetModuleDict(), "torch");
  PyObject* tensor = attribute(torch, "Tensor");
  PyObject* capsule = attribute(tensor, "__dlpack_c_exchange_api__");
  PyObject* c = attribute(torch, "_C");
  PyObject* device = attribute(c, "_cuda_getDevice");
  Py_XDECREF(c);
  if (capsule && device && PyType_Check(tensor) && PyCapsule_IsValid(capsule, "dlpack_exchange_api")) {
    const auto* api = static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
    if (api->header.version.major == DLPACK_MAJOR_VERSION && api->dltensor_from_py_object_no_sync && api->current_work_stream) {
      g_tensor = reinterpret_cast<PyTypeObject*>(tensor);
      g_device = device;
      g_api = api;
      return true;
    }
  }
  Py_XDECREF(device);
  Py_XDECREF(capsule);
  Py_XDECREF(tensor);
  return false;
}

bool contiguous(const DLTensor& t) {
  if (!t.strides) return true;
  for (int i = 0; i < t.ndim; ++i)
    if (t.shape[i] == 0) return true;
  int64_t step = 1;
  for (int i = t.ndim - 1; i >= 0; --i) {
    if (t.shape[i] != 1 && t.strides[i] != step) return false;
    step *= t.shape[i];
  }
  return true;
}

bool fits(unsigned holds, const DLDataType& t, const dsv4_moe_params& p, bool scaled) {
  if (t.lanes != 1) return false;
  if (holds == kRows) holds = scaled ? kE4m3 : kAct;
  if (holds == kAct || holds == kLogits) {
    const int32_t type = holds == kAct ? p.dtype : p.logits_dtype;
    if (type == DSV4_BF16) return t.code == kDLBfloat && t.bits == 16;
    holds = type == DSV4_F32 ? kF32 : kAny;  // another: for the function to refuse
  }
  if (holds == kF32) return t.code == kDLFloat && t.bits == 32;
  if (holds == kI32) return t.code == kDLInt && t.bits == 32;
  if (holds == kE4m3) return (t.code == kDLFloat8_e4m3fn || t.code == kDLUInt) && t.bits == 8;
  return true;
}

// Elements that the entry point of so many tensors reads and writes of the i-th; in floating point, which
// no sizes overflow.
double elements(int tensors, int i, const dsv4_moe_params& p) {
  const double T = p.T, rows = T * p.hidden, scales = T * ((p.hidden + 127LL) / 128), matrix = (double)p.E * p.inter * p.hidden;
  const double norm[] = {rows, rows, (double)p.hidden, rows, rows, rows, scales};
  const double route[] = {T * p.E, (double)p.E, T * p.topk, T * p.topk};
  const double experts[] = {rows, scales, T * p.topk, T * p.topk, 2 * matrix, matrix, rows, 0};
  return (tensors == 7 ? norm : tensors == 4 ? route : experts)[i];
}

// (params, tensor or None, ..., [handle of a stream or None]) -> status, or None: not for this way.
PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  const auto* e = static_cast<const Entry*>(PyCapsule_GetPointer(self, nullptr));
  if (!e) return nullptr;
  PyObject* given = n == e->tensors + 2 && args[n - 1] != Py_None ? args[n - 1] : nullptr;
  if ((n != e->tensors + 1 && n != e->tensors + 2) || (given && !PyLong_Check(given)) || !find_torch()) Py_RETURN_NONE;
  Py_buffer params;
  if (PyObject_GetBuffer(args[0], &params, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  dsv4_moe_params sizes;
  const bool right = params.len == (Py_ssize_t)sizeof(sizes);
  if (right) memcpy(&sizes, params.buf, sizeof(sizes));
  PyBuffer_Release(&params);
  if (!right) Py_RETURN_NONE;
  void* p[kMaxTensors];
  int device = -1;
  int64_t bytes = 0;
  for (int i = 0; i < e->tensors; ++i) {
    PyObject* o = args[i + 1];
    p[i] = nullptr;
    if (o == Py_None) continue;
    if (!PyObject_TypeCheck(o, g_tensor)) Py_RETURN_NONE;
    DLTensor t;
    if (g_api->dltensor_from_py_object_no_sync(o, &t) != 0) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (t.device.device_type != kDLCUDA || (device >= 0 && t.device.device_id != device) || !contiguous(t)) Py_RETURN_NONE;
    if (sizes.T > 0 && !fits((e->holds >> (4 * i)) & 15u, t.dtype, sizes, args[2] != Py_None)) Py_RETURN_NONE;
    int64_t n = 1;
    for (int j = 0; j < t.ndim; ++j) n *= t.shape[j];
    if (sizes.T > 0 && (double)n < elements(e->tensors, i, sizes)) Py_RETURN_NONE;
    device = t.device.device_id;
    p[i] = static_cast<char*>(t.data) + t.byte_offset;
    if (e->sized && i == e->tensors - 1) bytes = n * (t.dtype.bits * t.dtype.lanes / 8);
  }
  if (device < 0) Py_RETURN_NONE;
  PyObject* now = PyObject_CallNoArgs(g_device);
  if (!now) return nullptr;
  const long current = PyLong_AsLong(now);
  Py_DECREF(now);
  void* stream = nullptr;
  if (given) stream = PyLong_AsVoidPtr(given);
  if (current != device || PyErr_Occurred() || (!given && g_api->current_work_stream(kDLCUDA, device, &stream) != 0)) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  using V = void*;
  int status = 0;
  Py_BEGIN_ALLOW_THREADS
  if (e->tensors == 4)
    status = reinterpret_cast<int (*)(V, V, V, V, V, V)>(e->function)(&sizes, p[0], p[1], p[2], p[3], stream);
  else if (e->tensors == 7)
    status = reinterpret_cast<int (*)(V, V, V, V, V, V, V, V, V)>(e->function)(&sizes, p[0], p[1], p[2], p[3], p[4], p[5],
                                                                               p[6], stream);
  else
    status = reinterpret_cast<int (*)(V, V, V, V, V, V, V, V, V, size_t, V)>(e->function)(
        &sizes, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

void free_entry(PyObject* capsule) { delete static_cast<Entry*>(PyCapsule_GetPointer(capsule, nullptr)); }

PyMethodDef g_call = {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr};

// entry(address of the function, tensors, holds, sized) -> callable
PyObject* entry(PyObject*, PyObject* args) {
  unsigned long long address = 0;
  Entry e{};
  if (!PyArg_ParseTuple(args, "KiIi", &address, &e.tensors, &e.holds, &e.sized)) return nullptr;
  if (!address || (e.tensors != 4 && e.tensors != 7 && e.tensors != 8) || (e.sized != 0) != (e.tensors == 8)) {
    PyErr_SetString(PyExc_ValueError, "no entry point has these arguments");
    return nullptr;
  }
  e.function = reinterpret_cast<void*>(address);
  Entry* held = new Entry(e);
  PyObject* capsule = PyCapsule_New(held, nullptr, free_entry);
  if (!capsule) {
    delete held;
    return nullptr;
  }
  PyObject* f = PyCFunction_New(&g_call, capsule);
  Py_DECREF(capsule);
  return f;
}

PyMethodDef g_methods[] = {{"entry", entry, METH_VARARGS, "entry(address, tensors, holds, sized) -> callable"}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", "Calls of libdsv4 with tensors.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
