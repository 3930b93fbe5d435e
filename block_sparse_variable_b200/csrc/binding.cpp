// binding.cpp -- calls of the cache operators from Python.
//
// A decoding step makes these calls for a few microseconds of GPU work each,
// and describing a dozen tensors through ctypes takes longer than that (11 us
// of a 25 us call).  This module does only that part natively: it fills the
// bsa_tensor descriptors of include/bsa.h from torch tensors, checks their
// devices, finds the stream and the workspace, and calls the C entry that it
// is given the address of.  Nothing is kept between calls.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/bsa.h"

namespace {

constexpr int kMost = 12;  // tensors of a call

int dtype_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return BSA_F16;
    case at::kBFloat16: return BSA_BF16;
    case at::kFloat: return BSA_F32;
    case at::kUInt16: return BSA_U16;
    case at::kInt: return BSA_I32;
    case at::kLong: return BSA_I64;
    case at::kFloat8_e4m3fn: return BSA_F8E4M3;
    default: return 0;
  }
}

using T = const bsa_tensor *;
using P = const bsa_params *;

// the three entries and their workspace queries, by number of tensors and scalars
bsa_status query(int op, void *fn, T *t, P prm, const int64_t *x, size_t *n) {
  if (op == 0) return reinterpret_cast<decltype(&bsa_block_means_get_workspace)>(fn)(t[0], t[1], t[2], t[3], t[4], prm, t[5], n);
  if (op == 1)
    return reinterpret_cast<decltype(&bsa_select_blocks_get_workspace)>(fn)(t[0], t[1], t[2], t[3], t[4], prm, x[0], x[1], t[5], n);
  return reinterpret_cast<decltype(&bsa_decode_get_workspace)>(fn)(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], prm, t[9], t[10], n);
}
bsa_status run(int op, void *fn, T *t, P prm, const int64_t *x, void *ws, size_t n, void *s) {
  if (op == 0) return reinterpret_cast<decltype(&bsa_block_means)>(fn)(t[0], t[1], t[2], t[3], t[4], prm, t[5], ws, n, s);
  if (op == 1)
    return reinterpret_cast<decltype(&bsa_select_blocks)>(fn)(t[0], t[1], t[2], t[3], t[4], prm, x[0], x[1], t[5], ws, n, s);
  return reinterpret_cast<decltype(&bsa_decode)>(fn)(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], prm, t[9], t[10], ws, n, s);
}

constexpr int kTensors[3] = {6, 6, 11};

// call(op, entry, query_entry, params_bytes, tensors, (x0, x1), workspace or None, stream or None)
//   -> (status, True when the workspace query gave it, workspace)
PyObject *call(PyObject *, PyObject *args) {
  int op;
  unsigned long long fn, fn_query;
  Py_buffer prm;
  PyObject *tensors, *ws_obj, *stream_obj;
  int64_t x[2];
  if (!PyArg_ParseTuple(args, "iKKy*O!(LL)OO", &op, &fn, &fn_query, &prm, &PyTuple_Type, &tensors, &x[0], &x[1],
                        &ws_obj, &stream_obj))
    return nullptr;
  bsa_params params;
  const bool size_ok = size_t(prm.len) >= sizeof(params);
  if (size_ok) std::memcpy(&params, prm.buf, sizeof(params));
  PyBuffer_Release(&prm);
  if (!size_ok || op < 0 || op > 2 || PyTuple_GET_SIZE(tensors) != kTensors[op]) {
    PyErr_SetString(PyExc_ValueError, "bad call");
    return nullptr;
  }
  try {
    bsa_tensor desc[kMost];
    T ref[kMost];
    int device = -1;
    bool first = true;
    for (int i = 0; i < kTensors[op]; ++i) {
      PyObject *o = PyTuple_GET_ITEM(tensors, i);
      ref[i] = nullptr;
      if (o == Py_None) continue;
      if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected torch tensors");
        return nullptr;
      }
      const at::Tensor &t = THPVariable_Unpack(o);
      const int dev = t.is_cuda() ? int(t.get_device()) : -1;
      if (first) device = dev;
      first = false;
      if (dev != device || dev < 0) {
        PyErr_SetString(PyExc_ValueError, "all tensors must be on one CUDA device");
        return nullptr;
      }
      const int nd = int(t.dim());
      if (nd > 4) {
        PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
        return nullptr;
      }
      bsa_tensor &d = desc[i];
      std::memset(&d, 0, sizeof(d));
      d.data = t.numel() ? t.data_ptr() : nullptr;
      // an empty tensor may have no storage; nothing is read through it
      if (!t.numel()) d.data = reinterpret_cast<void *>(uintptr_t(256));
      d.dtype = dtype_of(t.scalar_type());
      d.ndim = nd;
      for (int k = 0; k < nd; ++k) {
        d.shape[k] = t.size(k);
        d.stride[k] = t.stride(k);
      }
      ref[i] = &d;
    }
    if (device < 0) {
      PyErr_SetString(PyExc_ValueError, "the tensors must be on a CUDA device");
      return nullptr;
    }
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    void *stream;
    if (stream_obj == Py_None) {
      stream = at::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    } else {
      stream = PyLong_AsVoidPtr(stream_obj);
      if (PyErr_Occurred()) return nullptr;
    }
    at::Tensor made;
    void *ws;
    size_t bytes = 0;
    if (ws_obj == Py_None) {
      const bsa_status st = query(op, reinterpret_cast<void *>(fn_query), ref, &params, x, &bytes);
      if (st != BSA_OK) return Py_BuildValue("(iOO)", int(st), Py_True, Py_None);
      if (bytes < 256) bytes = 256;
      // memory of the call's own stream: of another's it could be handed out
      // again while the kernels run
      c10::cuda::OptionalCUDAStreamGuard on;
      if (stream_obj != Py_None)
        on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                         static_cast<c10::DeviceIndex>(device)));
      made = at::empty({int64_t(bytes)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, device));
      ws = made.data_ptr();
    } else {
      if (!THPVariable_Check(ws_obj)) {
        PyErr_SetString(PyExc_TypeError, "the workspace must be a torch tensor");
        return nullptr;
      }
      const at::Tensor &t = THPVariable_Unpack(ws_obj);
      if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "the workspace must be a contiguous tensor on the tensors' device");
        return nullptr;
      }
      ws = t.numel() ? t.data_ptr() : nullptr;
      bytes = size_t(t.numel()) * t.element_size();
    }
    bsa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = run(op, reinterpret_cast<void *>(fn), ref, &params, x, ws, bytes, stream);
    Py_END_ALLOW_THREADS
    if (made.defined()) return Py_BuildValue("(iON)", int(st), Py_False, THPVariable_Wrap(made));
    return Py_BuildValue("(iOO)", int(st), Py_False, ws_obj);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {{"call", call, METH_VARARGS, "one call of a cache operator"}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
