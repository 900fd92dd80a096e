// The part of the binding that small steps cannot afford in Python: checks a list of tensors
// against a plan, collects their addresses and makes the library's call, in one native call.
// (GPT-2-124M's 122 vectors: the list's checks alone take 45 us from Python and 1 us here; the
// norm over them 12.5 us with the rest of the call in Python.) Errors are described in Python,
// from what these functions return.
//
// Host code only: built with the C++ compiler against PyTorch's headers. The library's functions
// come as addresses, so that nothing here binds to it.
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <vector>

namespace {

// muon_dtype of a tensor, 2 for codes and 3 for scales of 8-bit states, -1 for any other
int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return 0;
    case at::kFloat: return 1;
    case at::kFloat8_e4m3fn: return 2;
    case at::kFloat8_e8m0fnu: return 3;
    default: return -1;
  }
}

// (A lazily negated view's memory holds other values than the tensor.)
bool fits(const at::Tensor& t, int64_t numel, int dtype, long device) {
  return t.is_cuda() && t.get_device() == device && t.numel() == numel &&
         dtype_code(t) == dtype && t.is_contiguous() && !t.is_neg();
}

// A held buffer argument.
struct Buffer {
  Py_buffer view{};
  ~Buffer() {
    if (view.obj) PyBuffer_Release(&view);
  }
};

// A list or tuple of tensors beside the layout it has to have.
struct List {
  Buffer numels, dtypes;                         // int64 and muon_dtype as int32
  PyObject* items = nullptr;
  long device = 0;
  Py_ssize_t n = 0;
  ~List() { Py_XDECREF(items); }

  bool open(PyObject* tensors) {
    items = PySequence_Fast(tensors, "a list or tuple of tensors expected");
    if (!items) return false;
    n = PySequence_Fast_GET_SIZE(items);
    if (numels.view.len == n * 8 && dtypes.view.len == n * 4) return true;
    PyErr_SetString(PyExc_ValueError, "buffers and tensors differ in length");
    return false;
  }

  // Writes the addresses (None: 0). -1, or the index of the first entry that does not fit.
  Py_ssize_t addresses(uint64_t* to) const {
    PyObject** const list = PySequence_Fast_ITEMS(items);
    const int64_t* const numel = static_cast<const int64_t*>(numels.view.buf);
    const int32_t* const dtype = static_cast<const int32_t*>(dtypes.view.buf);
    for (Py_ssize_t i = 0; i < n; ++i) {
      if (list[i] == Py_None) {
        to[i] = 0;
        continue;
      }
      try {
        if (!THPVariable_Check(list[i])) return i;
        const at::Tensor& t = THPVariable_Unpack(list[i]);
        if (!fits(t, numel[i], dtype[i], device)) return i;
        to[i] = reinterpret_cast<uint64_t>(t.const_data_ptr());
        if (!to[i] && numel[i] > 0) return i;    // without storage: not one that is left out
      } catch (...) {                            // the same
        return i;
      }
    }
    return -1;
  }
};

// addresses(tensors, numels, dtypes, device, out) -> -1, or the index of the first entry that is
// neither None (address 0) nor a contiguous tensor of its size and dtype on the device.
PyObject* addresses(PyObject*, PyObject* args) {
  List list;
  Buffer out;
  PyObject* tensors;
  if (!PyArg_ParseTuple(args, "Oy*y*lw*", &tensors, &list.numels.view, &list.dtypes.view,
                        &list.device, &out.view) ||
      !list.open(tensors))
    return nullptr;
  if (out.view.len != list.n * 8) {
    PyErr_SetString(PyExc_ValueError, "buffers and tensors differ in length");
    return nullptr;
  }
  return PyLong_FromSsize_t(list.addresses(static_cast<uint64_t*>(out.view.buf)));
}

// entries_at(dicts, keys, addresses) -> whether the tensors under `keys` (a tuple) in each of a list
// of dicts are at the addresses, dict by dict; 0: no such entry, or one without memory.
PyObject* entries_at(PyObject*, PyObject* args) {
  PyObject *dicts, *keys;
  Buffer at;
  if (!PyArg_ParseTuple(args, "O!O!y*", &PyList_Type, &dicts, &PyTuple_Type, &keys, &at.view))
    return nullptr;
  const Py_ssize_t n = PyList_GET_SIZE(dicts), k = PyTuple_GET_SIZE(keys);
  if (at.view.len != n * k * 8) {
    PyErr_SetString(PyExc_ValueError, "addresses and entries differ in length");
    return nullptr;
  }
  const uint64_t* want = static_cast<const uint64_t*>(at.view.buf);
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const dict = PyList_GET_ITEM(dicts, i);
      if (!PyDict_Check(dict)) Py_RETURN_FALSE;
      for (Py_ssize_t j = 0; j < k; ++j, ++want) {
        PyObject* const t = PyDict_GetItemWithError(dict, PyTuple_GET_ITEM(keys, j));
        if (!t && PyErr_Occurred()) return nullptr;
        const uint64_t is = t && THPVariable_Check(t)
            ? reinterpret_cast<uint64_t>(THPVariable_Unpack(t).const_data_ptr()) : 0;
        if (is != *want) Py_RETURN_FALSE;
      }
    }
  } catch (const std::exception&) {              // a tensor without storage
    Py_RETURN_FALSE;
  }
  Py_RETURN_TRUE;
}

// A step's arguments, given to muon_adamw_step, or without a stream to muon_adamw_check.
PyObject* adamw_call(PyObject* args, bool step) {
  List list;
  Buffer cfg;
  PyObject *tensors, *scale;
  unsigned long long function, plan, stream = 0;
  Py_ssize_t offset;
  if (!PyArg_ParseTuple(args, step ? "KKOy*y*ly*OnK" : "KKOy*y*ly*On", &function, &plan, &tensors,
                        &list.numels.view, &list.dtypes.view, &list.device, &cfg.view, &scale,
                        &offset, &stream) ||
      !list.open(tensors))
    return nullptr;
  try {
    std::vector<uint64_t> grads(list.n);
    const Py_ssize_t bad = list.addresses(grads.data());
    if (bad >= 0) return PyLong_FromSsize_t(bad);
    alignas(16) char config[256];
    const Py_ssize_t size = cfg.view.len;
    if (size > Py_ssize_t(sizeof config) || offset < 0 || offset + 8 > size) {
      PyErr_SetString(PyExc_ValueError, "not a step's configuration");
      return nullptr;
    }
    std::memcpy(config, cfg.view.buf, size);
    if (scale != Py_None) {
      const void* at = nullptr;
      if (THPVariable_Check(scale) && fits(THPVariable_Unpack(scale), 1, 1, list.device))
        at = THPVariable_Unpack(scale).const_data_ptr();
      if (!at) {
        PyErr_SetString(PyExc_ValueError, "grad_scale must be one float32 on the plan's device");
        return nullptr;
      }
      std::memcpy(config + offset, &at, sizeof at);
    }
    typedef int (*Step)(const void*, const void*, int64_t, const void*, void*);
    typedef int (*Check)(const void*, const void*, int64_t, const void*);
    const void* const p = reinterpret_cast<const void*>(plan);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = step ? reinterpret_cast<Step>(function)(p, grads.data(), list.n, config,
                                                     reinterpret_cast<void*>(stream))
                  : reinterpret_cast<Check>(function)(p, grads.data(), list.n, config);
    Py_END_ALLOW_THREADS
    if (status) return PyLong_FromLong(status);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// adamw_step(function, plan, tensors, numels, dtypes, device, cfg, scale, offset, stream) -> None,
// the index (>= 0) of a gradient that does not fit, or the library's status (< 0). scale: None, or
// one float32 on the device, whose address goes into the copy of cfg at `offset`.
PyObject* adamw_step(PyObject*, PyObject* args) { return adamw_call(args, true); }

// adamw_check: the same without `stream`, and without the step.
PyObject* adamw_check(PyObject*, PyObject* args) { return adamw_call(args, false); }

// grad_norm(function, plan, tensors, numels, dtypes, device, max_norm, per_tensor, workspace_bytes,
// stream) -> (norm, scale) or (norm, scale, norms), or as adamw_step. Results and workspace are new
// allocations of the current stream: a workspace over kShared bytes one of its own, so that results
// that a caller keeps, a norm of each step, do not hold it, a smaller one behind the results (16-byte
// aligned), since the second allocation takes 0.6 us of a call of 10 (122 vectors).
constexpr Py_ssize_t kShared = 4096;

PyObject* grad_norm(PyObject*, PyObject* args) {
  List list;
  PyObject* tensors;
  unsigned long long function, plan, stream;
  float max_norm;
  int per_tensor;
  Py_ssize_t ws_bytes;
  if (!PyArg_ParseTuple(args, "KKOy*y*lfpnK", &function, &plan, &tensors, &list.numels.view,
                        &list.dtypes.view, &list.device, &max_norm, &per_tensor, &ws_bytes,
                        &stream) ||
      !list.open(tensors))
    return nullptr;
  try {
    std::vector<uint64_t> grads(list.n);
    const Py_ssize_t bad = list.addresses(grads.data());
    if (bad >= 0) return PyLong_FromSsize_t(bad);
    const int64_t each = per_tensor ? list.n : 0, ws = (2 + each + 3) / 4 * 4;
    const int64_t ws_floats = (ws_bytes + 3) / 4;
    const bool shared = ws_bytes <= kShared;
    const auto options =
        at::TensorOptions().dtype(at::kFloat).device(at::kCUDA, c10::DeviceIndex(list.device));
    const at::Tensor out = at::empty({shared ? ws + ws_floats : 2 + each}, options);
    const at::Tensor own = shared ? at::Tensor() : at::empty({ws_floats}, options);
    float* const base = static_cast<float*>(out.data_ptr());
    void* const workspace = shared ? base + ws : own.data_ptr();
    typedef int (*Norm)(const void*, const void*, int64_t, float, float*, float*, void*, size_t,
                        void*);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Norm>(function)(
        reinterpret_cast<const void*>(plan), grads.data(), list.n, max_norm, base,
        each ? base + 2 : nullptr, workspace, size_t(ws_bytes),
        reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (status) return PyLong_FromLong(status);
    PyObject* const result = PyTuple_New(per_tensor ? 3 : 2);
    if (!result) return nullptr;
    PyTuple_SET_ITEM(result, 0, THPVariable_Wrap(out.select(0, 0)));
    PyTuple_SET_ITEM(result, 1, THPVariable_Wrap(out.select(0, 1)));
    if (per_tensor) PyTuple_SET_ITEM(result, 2, THPVariable_Wrap(out.narrow(0, 2, each)));
    return result;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"addresses", addresses, METH_VARARGS, "Addresses of the tensors of a plan's layout."},
    {"entries_at", entries_at, METH_VARARGS, "Whether dicts hold tensors at these addresses."},
    {"adamw_step", adamw_step, METH_VARARGS, "muon_adamw_step over a list of gradients."},
    {"adamw_check", adamw_check, METH_VARARGS, "muon_adamw_check over a list of gradients."},
    {"grad_norm", grad_norm, METH_VARARGS, "muon_grad_norm over a list of gradients."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
