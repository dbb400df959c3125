// marshal.cpp -- the Python binding's argument marshalling for the feed-forward
// operators (module _marshal): tensors, addresses and numbers into the
// descriptors of igc.h, and the call.  A small call takes a few microseconds
// on the GPU; filling a ctypes structure for it takes five (grad_clip of 40
// tensors, one Python call per property of each: 37).
#include <Python.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <exception>
#include <vector>

#include "../../include/igc.h"

namespace {

// What a Python argument stands for as a device address: None, an int, a
// tensor, or anything with data_ptr().
bool address(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  if (THPVariable_Check(o)) {
    *out = THPVariable_Unpack(o).data_ptr();
    return true;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  if (!PyObject_HasAttrString(o, "data_ptr")) {
    PyErr_Format(PyExc_TypeError, "expected a device address or a tensor, got %R", (PyObject*)Py_TYPE(o));
    return false;
  }
  PyObject* const r = PyObject_CallMethod(o, "data_ptr", nullptr);
  if (!r) return false;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

bool integer(PyObject* o, int* out) {
  PyObject* const n = PyNumber_Index(o);
  if (!n) return false;
  const long v = PyLong_AsLong(n);
  Py_DECREF(n);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_Format(PyExc_OverflowError, "%ld does not fit in 32 bits", v);
    return false;
  }
  *out = (int)v;
  return true;
}

// The workspace's address and, where the caller gives no size, its bytes.
bool workspace(PyObject* ws, PyObject* bytes, void** p, size_t* size) {
  if (!address(ws, p)) return false;
  *size = 0;
  if (bytes != Py_None) {
    *size = PyLong_AsSize_t(bytes);
    return !PyErr_Occurred();
  }
  if (THPVariable_Check(ws)) *size = THPVariable_Unpack(ws).nbytes();
  return true;
}

// C++ exceptions (a tensor without storage) end here.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The call, without the interpreter's lock (a full queue makes a launch wait).
int enter(void* entry, const void* descriptor, void* second) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = reinterpret_cast<int (*)(const void*, void*)>(entry)(descriptor, second);
  Py_END_ALLOW_THREADS
  return status;
}

// call(entry, format, stream, ws, ws_bytes, fields...) -> status.  The
// descriptor is laid out as the C compiler does: "i" an int, "p" an address;
// the workspace and its size come last.
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n < 5) return PyErr_Format(PyExc_TypeError, "call takes at least 5 arguments, not %zd", n);
    void *entry, *stream;
    if (!address(args[0], &entry) || !address(args[2], &stream)) return nullptr;
    Py_ssize_t fields;
    const char* const format = PyUnicode_AsUTF8AndSize(args[1], &fields);
    if (!format) return nullptr;
    alignas(8) unsigned char d[512] = {};
    if (!entry || fields != n - 5 || fields * 8 + 16 > (Py_ssize_t)sizeof(d))
      return PyErr_Format(PyExc_TypeError, "%zd fields for the format %s", n - 5, format);
    size_t at = 0;
    for (Py_ssize_t i = 0; i < fields; ++i) {
      if (format[i] == 'i') {
        int v;
        if (!integer(args[5 + i], &v)) return nullptr;
        std::memcpy(d + at, &v, 4);
        at += 4;
      } else {
        void* p;
        if (!address(args[5 + i], &p)) return nullptr;
        at = (at + 7) & ~size_t(7);
        std::memcpy(d + at, &p, 8);
        at += 8;
      }
    }
    void* ws;
    size_t size;
    if (!workspace(args[3], args[4], &ws, &size)) return nullptr;
    at = (at + 7) & ~size_t(7);
    std::memcpy(d + at, &ws, 8);
    std::memcpy(d + at + 8, &size, 8);
    return PyLong_FromLong(enter(entry, d, stream));
  });
}

// The tensors of a sequence.
struct Tensors {
  PyObject* fast = nullptr;
  Py_ssize_t n = 0;
  ~Tensors() { Py_XDECREF(fast); }
  bool open(PyObject* seq) {
    fast = PySequence_Fast(seq, "grad_clip takes sequences of tensors");
    if (!fast) return false;
    n = PySequence_Fast_GET_SIZE(fast);
    return true;
  }
  // NULL with a Python error: no tensor, or not contiguous
  const at::Tensor* operator()(Py_ssize_t i) const {
    PyObject* const o = PySequence_Fast_GET_ITEM(fast, i);
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "grad_clip takes tensors, not %R", (PyObject*)Py_TYPE(o));
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "grad_clip takes contiguous tensors");
      return nullptr;
    }
    return &t;
  }
};

// The kernels take addresses of the current device only; with a Python error,
// false for a tensor of another.  (`current` is asked for once a call.)
bool on_device(const at::Tensor& t, c10::Device& current) {
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_TypeError, "grad_clip takes tensors on the GPU, not on %s", t.device().str().c_str());
    return false;
  }
  if (!current.is_cuda()) current = c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice();
  if (t.device() == current) return true;
  PyErr_Format(PyExc_ValueError, "a tensor on %s in a call on %s", t.device().str().c_str(), current.str().c_str());
  return false;
}

// clip(entry, query, stream, ws, ws_bytes, grads, outs or None, max_norm, norm)
// -> status, or with query (status, bytes).
PyObject* clip(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) return PyErr_Format(PyExc_TypeError, "clip takes 9 arguments, not %zd", n);
    void *entry, *stream, *norm, *ws;
    size_t size;
    const int query = PyObject_IsTrue(args[1]);
    const double max_norm = PyFloat_AsDouble(args[7]);
    if (query < 0 || PyErr_Occurred()) return nullptr;
    if (!address(args[0], &entry) || !address(args[2], &stream) || !address(args[8], &norm) || !workspace(args[3], args[4], &ws, &size))
      return nullptr;
    const bool out = args[6] != Py_None;
    Tensors grads, outs;
    if (!grads.open(args[5]) || (out && !outs.open(args[6]))) return nullptr;
    if (out && outs.n != grads.n)
      return PyErr_Format(PyExc_ValueError, "%zd gradients but %zd outputs", grads.n, outs.n);
    if (grads.n > INT_MAX) return PyErr_Format(PyExc_OverflowError, "too many tensors");
    std::vector<const void*> from(grads.n);
    std::vector<void*> to(out ? grads.n : 0);
    std::vector<long long> sizes(grads.n);
    std::vector<int> types(grads.n);
    for (Py_ssize_t i = 0; i < grads.n; ++i) {
      const at::Tensor* const g = grads(i);
      if (!g) return nullptr;
      switch (g->scalar_type()) {
        case at::kHalf: types[i] = IGC_F16; break;
        case at::kBFloat16: types[i] = IGC_BF16; break;
        case at::kFloat: types[i] = IGC_F32; break;
        default: {
          PyObject* const dtype = PyObject_GetAttrString(PySequence_Fast_GET_ITEM(grads.fast, i), "dtype");
          if (dtype) PyErr_Format(PyExc_TypeError, "grad_clip takes float16, bfloat16 and float32 tensors, not %S", dtype);
          Py_XDECREF(dtype);
          return nullptr;
        }
      }
      from[i] = g->data_ptr();
      sizes[i] = g->numel();
      if (!out) continue;
      const at::Tensor* const o = outs(i);
      if (!o) return nullptr;
      if (o->scalar_type() != g->scalar_type() || o->numel() != g->numel()) {
        PyErr_SetString(PyExc_ValueError, "an output differs from its gradient in type or size");
        return nullptr;
      }
      to[i] = o->data_ptr();
    }
    if (THPVariable_Check(args[8])) {
      const at::Tensor& t = THPVariable_Unpack(args[8]);
      if (t.scalar_type() != at::kFloat || t.numel() < 1)
        return PyErr_Format(PyExc_TypeError, "norm must be a float32 tensor of one element");
    }
    if (!query) {
      c10::Device current(c10::DeviceType::CPU);
      for (Py_ssize_t i = 0; i < grads.n; ++i)
        if (!on_device(*grads(i), current) || (out && !on_device(*outs(i), current))) return nullptr;
      for (PyObject* const o : {args[8], args[3]})
        if (THPVariable_Check(o) && !on_device(THPVariable_Unpack(o), current)) return nullptr;
    }
    igc_grad_clip d;
    std::memset(&d, 0, sizeof(d));
    d.count = (int)grads.n;
    d.grads = from.data();
    d.outs = out ? to.data() : nullptr;
    d.sizes = sizes.data();
    d.types = types.data();
    d.max_norm = (float)max_norm;
    d.norm = static_cast<float*>(norm);
    d.workspace = ws;
    d.ws_bytes = size;
    if (!query) return PyLong_FromLong(enter(entry, &d, stream));
    size_t bytes = 0;
    const int status = enter(entry, &d, &bytes);
    return Py_BuildValue("in", status, (Py_ssize_t)bytes);
  });
}

PyMethodDef methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr},
    {"clip", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(clip)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
