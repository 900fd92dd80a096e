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
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
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

// ---- microscaled 4-bit values (include/mx4.h) ----

// muon_mx_source, for calls through an address.
struct MxSource {
  const void* x;
  int64_t rows, cols, row_stride;
  int dtype;
  void *codes, *scales, *codes_t, *scales_t;
};

int64_t mx_codes(int64_t rows, int64_t cols) { return (rows + 15) / 16 * ((cols + 127) / 128) * 1024; }

// Whether t is rows of its last dimension: its leading dimensions collapse into rows of one stride and
// the last has stride 1, or (transposed) it is 2-D and its transpose is.
bool rows_of(const at::Tensor& t, MxSource& s, bool& transposed) {
  const auto size = t.sizes(), stride = t.strides();
  const int64_t d = t.dim();
  transposed = false;
  if (d == 0) return false;
  s.cols = size[d - 1];
  s.rows = 1;
  s.row_stride = s.cols;
  bool first = true, fits = s.cols <= 1 || stride[d - 1] == 1;
  for (int64_t i = d - 2; i >= 0; --i) {
    if (size[i] != 1) {
      if (first) s.row_stride = stride[i];
      else fits = fits && stride[i] == s.row_stride * s.rows;
      first = false;
    }
    s.rows *= size[i];
  }
  if (t.numel() == 0 || (fits && (s.rows <= 1 || s.row_stride >= s.cols))) return true;
  if (d != 2 || stride[0] != 1 || stride[1] < size[0]) return false;
  transposed = true;
  s.rows = size[1];
  s.cols = size[0];
  s.row_stride = stride[1];
  return true;
}

// What a native call returns to Python for a refused argument; the text is the error's.
PyObject* refuse(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  return nullptr;
}

// mx_quantize(function, tensors, results, stochastic, seed, stream) -> for each tensor (rows, cols,
// data, data_t), rows x cols the matrix that it is as rows of its last dimension, data and data_t the
// held form of that and of its transpose, codes and then scales in one uint8 tensor (None where
// `results`, a bytes of 1: rows, 2: transposed, 3: both for each tensor, does not ask for it); or the
// library's status.
PyObject* mx_quantize(PyObject*, PyObject* args) {
  PyObject* tensors;
  Buffer results;
  unsigned long long function, seed, stream;
  int stochastic;
  if (!PyArg_ParseTuple(args, "KOy*pKK", &function, &tensors, &results.view, &stochastic, &seed,
                        &stream))
    return nullptr;
  if (!PyTuple_Check(tensors) || PyTuple_GET_SIZE(tensors) != results.view.len)
    return refuse(PyExc_ValueError, "a tuple of tensors and a result kind for each expected");
  const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
  const char* const kinds = static_cast<const char*>(results.view.buf);
  try {
    std::vector<MxSource> sources(n);
    std::vector<at::Tensor> out(2 * n);
    std::vector<bool> turned(n);
    c10::OptionalDeviceGuard guard;
    long device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const o = PyTuple_GET_ITEM(tensors, i);
      if (!THPVariable_Check(o)) return refuse(PyExc_TypeError, "a tensor expected");
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cuda() || t.layout() != at::kStrided)
        return refuse(PyExc_ValueError, "a CUDA tensor expected");
      if (dtype_code(t) != 0 && dtype_code(t) != 1)
        return refuse(PyExc_TypeError, "unsupported dtype: the library takes bfloat16 or float32");
      if (device < 0) {
        device = t.get_device();
        guard.reset_device(t.device());
      }
      MxSource& s = sources[i];
      bool transposed = false;
      if (t.get_device() != device || t.is_neg() || !rows_of(t, s, transposed))
        return refuse(PyExc_ValueError, t.get_device() != device
                          ? "all tensors must be on one device"
                          : "rows of the last dimension expected: a tensor with stride 1 there (or, in "
                            "two dimensions, along the other) and one stride between rows");
      s.x = t.numel() ? t.const_data_ptr() : nullptr;
      if (!s.x && t.numel()) return refuse(PyExc_ValueError, "a tensor with memory expected");
      s.dtype = dtype_code(t);
      turned[i] = transposed;
      s.codes = s.scales = s.codes_t = s.scales_t = nullptr;
      if (s.rows > (int64_t(1) << 31) || s.cols > (int64_t(1) << 31))
        return refuse(PyExc_ValueError, "sides up to 2^31 - 256");
      const auto options = at::TensorOptions().dtype(at::kByte).device(t.device());
      for (int k = 0; k < 2; ++k) {              // 0: as it is in memory, 1: the transpose of that
        if (!(kinds[i] & ((k == 1) != transposed ? 2 : 1))) continue;
        const int64_t codes = k ? mx_codes(s.cols, s.rows) : mx_codes(s.rows, s.cols);
        at::Tensor& d = out[2 * i + ((k == 1) != transposed ? 1 : 0)];
        d = at::empty({codes / 16 * 17}, options);
        char* const p = static_cast<char*>(d.data_ptr());
        (k ? s.codes_t : s.codes) = p;
        (k ? s.scales_t : s.scales) = p ? p + codes : nullptr;
      }
    }
    typedef int (*Quantize)(const void*, int64_t, int, uint64_t, void*);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Quantize>(function)(sources.data(), n, stochastic, seed,
                                                  reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (status) return PyLong_FromLong(status);
    PyObject* const result = PyTuple_New(n);
    if (!result) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
      const MxSource& s = sources[i];
      PyObject* const each =
          Py_BuildValue("LLNN", (long long)(turned[i] ? s.cols : s.rows),
                        (long long)(turned[i] ? s.rows : s.cols), THPVariable_Wrap(out[2 * i]),
                        THPVariable_Wrap(out[2 * i + 1]));
      if (!each) {
        Py_DECREF(result);
        return nullptr;
      }
      PyTuple_SET_ITEM(result, i, each);
    }
    return result;
  } catch (const std::exception& e) {
    return refuse(PyExc_RuntimeError, e.what());
  }
}

// The held form in `o`: a uint8 tensor of the size that rows x cols take. Null with an error set.
const char* held(PyObject* o, int64_t rows, int64_t cols, at::Device* device) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.is_cuda() && t.scalar_type() == at::kByte && t.is_contiguous() &&
        t.numel() == mx_codes(rows, cols) / 16 * 17 && (!device->has_index() || t.device() == *device)) {
      *device = t.device();
      static const char empty = 0;
      return t.numel() ? static_cast<const char*>(t.const_data_ptr()) : &empty;
    }
  }
  PyErr_SetString(PyExc_ValueError, "held values of these sizes, on one device, expected");
  return nullptr;
}

at::ScalarType out_type(int dtype) { return dtype ? at::kFloat : at::kBFloat16; }

// mx_dequantize(function, data, rows, cols, dtype, stream) -> a rows x cols tensor, or the status.
PyObject* mx_dequantize(PyObject*, PyObject* args) {
  PyObject* data;
  unsigned long long function, stream;
  long long rows, cols;
  int dtype;
  if (!PyArg_ParseTuple(args, "KOLLiK", &function, &data, &rows, &cols, &dtype, &stream))
    return nullptr;
  try {
    at::Device device(at::kCUDA);
    const char* const p = held(data, rows, cols, &device);
    if (!p) return nullptr;
    const c10::DeviceGuard guard(device);
    const at::Tensor out =
        at::empty({rows, cols}, at::TensorOptions().dtype(out_type(dtype)).device(device));
    typedef int (*Back)(const void*, const void*, int64_t, int64_t, void*, int, void*);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Back>(function)(p, p + mx_codes(rows, cols), rows, cols,
                                              out.data_ptr(), dtype,
                                              reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    return status ? PyLong_FromLong(status) : THPVariable_Wrap(out);
  } catch (const std::exception& e) {
    return refuse(PyExc_RuntimeError, e.what());
  }
}

// mx_matmul(function, workspace_size, a, b, m, n, k, dtype, stream) -> an m x n tensor, or the status.
PyObject* mx_matmul(PyObject*, PyObject* args) {
  PyObject *a, *b;
  unsigned long long function, size, stream;
  long long m, n, k;
  int dtype;
  if (!PyArg_ParseTuple(args, "KKOOLLLiK", &function, &size, &a, &b, &m, &n, &k, &dtype, &stream))
    return nullptr;
  try {
    at::Device device(at::kCUDA);
    const char* const p = held(a, m, k, &device);
    const char* const q = p ? held(b, n, k, &device) : nullptr;
    if (!q) return nullptr;
    const c10::DeviceGuard guard(device);
    const at::Tensor out =
        at::empty({m, n}, at::TensorOptions().dtype(out_type(dtype)).device(device));
    typedef size_t (*Size)(int64_t, int64_t, int64_t);
    const size_t need = reinterpret_cast<Size>(size)(m, n, k);
    at::Tensor ws;
    if (need && need != SIZE_MAX)
      ws = at::empty({int64_t(need)}, at::TensorOptions().dtype(at::kByte).device(device));
    typedef int (*Product)(const void*, const void*, const void*, const void*, int64_t, int64_t,
                           int64_t, void*, int, void*, size_t, void*);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Product>(function)(
        p, p + mx_codes(m, k), q, q + mx_codes(n, k), m, n, k, out.data_ptr(), dtype,
        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? need : 0,
        reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    return status ? PyLong_FromLong(status) : THPVariable_Wrap(out);
  } catch (const std::exception& e) {
    return refuse(PyExc_RuntimeError, e.what());
  }
}

// ---- orthogonalisation of stacks (include/orthogonalize.h) ----

// muon_stack, for calls through an address.
struct Stack {
  const void* in;
  void* out;
  int64_t side[4];
  int64_t in_stride[4], out_stride[4];
  int dtype;
};

// orthogonalize(function, workspace_size, x, out, cfg, stream) -> out (a new tensor in x's order of
// strides where it is None), or the status. x: at least 2-D, its leading dimensions two strides at
// most.
PyObject* orthogonalize(PyObject*, PyObject* args) {
  PyObject *xo, *oo;
  Buffer cfg;
  unsigned long long function, size, stream;
  if (!PyArg_ParseTuple(args, "KKOOy*K", &function, &size, &xo, &oo, &cfg.view, &stream))
    return nullptr;
  if (!THPVariable_Check(xo) || (oo != Py_None && !THPVariable_Check(oo)))
    return refuse(PyExc_TypeError, "tensors expected");
  try {
    const at::Tensor& x = THPVariable_Unpack(xo);
    if (!x.is_cuda() || x.layout() != at::kStrided || x.is_neg())
      return refuse(PyExc_ValueError, "a CUDA tensor whose memory holds its values expected");
    if (dtype_code(x) != 0 && dtype_code(x) != 1)
      return refuse(PyExc_TypeError, "unsupported dtype: the library takes bfloat16 or float32");
    const int64_t d = x.dim();
    if (d < 2) return refuse(PyExc_ValueError, "a matrix or a stack of them expected");
    const c10::DeviceGuard guard(x.device());
    at::Tensor out;
    if (oo == Py_None) {                         // dense, dimensions in x's order of strides
      std::vector<int64_t> order(d), strides(d);
      for (int64_t i = 0; i < d; ++i) order[i] = i;
      auto far = [&](int64_t i) {                // (a dimension without strides goes outside)
        return x.size(i) > 1 && x.stride(i) == 0 ? INT64_MAX : x.stride(i);
      };
      std::stable_sort(order.begin(), order.end(), [&](int64_t a, int64_t b) { return far(a) > far(b); });
      int64_t step = 1;
      for (int64_t i = d; i-- > 0;) {
        strides[order[i]] = step;
        step *= std::max<int64_t>(x.size(order[i]), 1);
      }
      out = at::empty_strided(x.sizes(), strides, x.options().requires_grad(false));
    } else {
      out = THPVariable_Unpack(oo);
      if (out.device() != x.device() || out.scalar_type() != x.scalar_type() ||
          out.sizes() != x.sizes() || out.layout() != at::kStrided || out.is_neg())
        return refuse(PyExc_ValueError, "out must be a tensor of x's shape, dtype and device");
    }
    Stack k{};
    k.dtype = dtype_code(x);
    k.in = x.numel() ? x.const_data_ptr() : nullptr;
    k.out = x.numel() ? out.data_ptr() : nullptr;
    // leading dimensions, from the last: each joins the group behind it or opens the next one outside
    int64_t sides[2] = {1, 1}, si[2] = {0, 0}, so[2] = {0, 0};
    int groups = 0;
    for (int64_t i = d - 3; i >= 0; --i) {
      const int64_t n = x.size(i);
      if (n == 1) continue;
      if (groups && x.stride(i) == si[groups - 1] * sides[groups - 1] &&
          out.stride(i) == so[groups - 1] * sides[groups - 1]) {
        sides[groups - 1] *= n;
        continue;
      }
      if (groups == 2)
        return refuse(PyExc_ValueError, "leading dimensions of more than two strides");
      sides[groups] = n;
      si[groups] = x.stride(i);
      so[groups] = out.stride(i);
      ++groups;
    }
    for (int j = 0; j < 2; ++j) {                // group 0 is the inner one
      k.side[1 - j] = sides[j];
      k.in_stride[1 - j] = si[j];
      k.out_stride[1 - j] = so[j];
      k.side[2 + j] = x.size(d - 2 + j);
      k.in_stride[2 + j] = x.stride(d - 2 + j);
      k.out_stride[2 + j] = out.stride(d - 2 + j);
    }
    typedef size_t (*Size)(int64_t, int64_t, int64_t, int64_t);
    const size_t need = reinterpret_cast<Size>(size)(k.side[0], k.side[1], k.side[2], k.side[3]);
    at::Tensor ws;
    if (need && need != SIZE_MAX)
      ws = at::empty({int64_t(need)}, at::TensorOptions().dtype(at::kByte).device(x.device()));
    typedef int (*Run)(const void*, const void*, void*, size_t, void*);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Run>(function)(&k, cfg.view.buf, ws.defined() ? ws.data_ptr() : nullptr,
                                             ws.defined() ? need : 0, reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    return status ? PyLong_FromLong(status) : THPVariable_Wrap(out);
  } catch (const std::exception& e) {
    return refuse(PyExc_RuntimeError, e.what());
  }
}

PyMethodDef methods[] = {
    {"orthogonalize", orthogonalize, METH_VARARGS, "muon_orthogonalize of a stack."},
    {"mx_quantize", mx_quantize, METH_VARARGS, "muon_mx_quantize of tensors into new ones."},
    {"mx_dequantize", mx_dequantize, METH_VARARGS, "muon_mx_dequantize into a new tensor."},
    {"mx_matmul", mx_matmul, METH_VARARGS, "muon_mx_matmul into a new tensor."},
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
