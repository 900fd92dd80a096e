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
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <memory>
#include <stdexcept>
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

// ---- the library's functions that are called without a plan ----

typedef int (*Quantize)(const void*, int64_t, int, uint64_t, void*);
typedef int (*Dequantize)(const void*, const void*, int64_t, int64_t, void*, int, void*);
typedef int (*Product)(const void*, const void*, const void*, const void*, int64_t, int64_t, int64_t, void*,
                       int, void*, size_t, void*);
typedef size_t (*ProductSize)(int64_t, int64_t, int64_t);
typedef int (*Stacked)(const void*, const void*, void*, size_t, void*);
typedef size_t (*StackedSize)(int64_t, int64_t, int64_t, int64_t);
typedef int (*Passes)(const void*);
typedef const char* (*LastError)();

struct Library {
  Quantize quantize;
  Dequantize dequantize;
  Product product;
  ProductSize product_size;
  Stacked stacked;
  StackedSize stacked_size;
  Passes passes;
  LastError last_error;
} library;

// bind(quantize, dequantize, matmul, its workspace, orthogonalize, its workspace, its passes, last error):
// their addresses, before any of the calls below.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[8];
  if (!PyArg_ParseTuple(args, "KKKKKKKK", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7)) return nullptr;
  library = {reinterpret_cast<Quantize>(f[0]),  reinterpret_cast<Dequantize>(f[1]),
             reinterpret_cast<Product>(f[2]),   reinterpret_cast<ProductSize>(f[3]),
             reinterpret_cast<Stacked>(f[4]),   reinterpret_cast<StackedSize>(f[5]),
             reinterpret_cast<Passes>(f[6]),    reinterpret_cast<LastError>(f[7])};
  Py_RETURN_NONE;
}

void* stream_of(const at::Device& device) {
  return static_cast<void*>(c10::hip::getCurrentHIPStream(device.index()).stream());
}

// Why a call was not made: an argument that does not fit, or the library's status.
struct Refused {
  PyObject* type;
  const char* text;
};
struct Failed {
  int status;
};

void check(int status) {
  if (status) throw Failed{status};
}

// What a native call returns to Python: f's result, the library's status as an int, or an error.
template <typename F>
PyObject* answer(F&& f) {
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text);
  } catch (const Failed& e) {
    return PyLong_FromLong(e.status);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// Runs f without the interpreter's lock.
template <typename F>
auto unlocked(F&& f) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
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

// A tensor as rows x cols, and the held form of that and of its transpose, codes and then scales in one
// uint8 tensor (undefined where not asked for).
struct Held {
  int64_t rows = 0, cols = 0;
  at::Tensor data, data_t;
};

// kinds: of each tensor 1: rows, 2: transposed, 3: both.
void quantize(const at::Tensor* const* tensors, const char* kinds, Held* out, int64_t n, bool stochastic,
              uint64_t seed) {
  std::vector<MxSource> sources(n);
  if (n == 0) return;
  for (int64_t i = 0; i < n; ++i) {
    const at::Tensor& t = *tensors[i];
    if (!t.is_cuda() || t.layout() != at::kStrided)
      throw Refused{PyExc_ValueError, "a CUDA tensor expected"};
    if (dtype_code(t) != 0 && dtype_code(t) != 1)
      throw Refused{PyExc_TypeError, "unsupported dtype: the library takes bfloat16 or float32"};
    if (t.device() != tensors[0]->device())
      throw Refused{PyExc_ValueError, "all tensors must be on one device"};
  }
  const at::Device device = tensors[0]->device();
  const c10::DeviceGuard guard(device);
  for (int64_t i = 0; i < n; ++i) {
    const at::Tensor& t = *tensors[i];
    MxSource& s = sources[i];
    bool turned = false;
    if (t.is_neg() || !rows_of(t, s, turned))
      throw Refused{PyExc_ValueError,
                    "rows of the last dimension expected: a tensor with stride 1 there (or, in two "
                    "dimensions, along the other) and one stride between rows"};
    s.x = t.numel() ? t.const_data_ptr() : nullptr;
    if (!s.x && t.numel()) throw Refused{PyExc_ValueError, "a tensor with memory expected"};
    s.dtype = dtype_code(t);
    s.codes = s.scales = s.codes_t = s.scales_t = nullptr;
    if (s.rows > (int64_t(1) << 31) || s.cols > (int64_t(1) << 31))
      throw Refused{PyExc_ValueError, "sides up to 2^31 - 256"};
    const auto options = at::TensorOptions().dtype(at::kByte).device(device);
    for (int k = 0; k < 2; ++k) {                // 0: as it is in memory, 1: the transpose of that
      const bool of_t = (k == 1) != turned;
      if (!(kinds[i] & (of_t ? 2 : 1))) continue;
      const int64_t codes = k ? mx_codes(s.cols, s.rows) : mx_codes(s.rows, s.cols);
      const at::Tensor d = at::empty({codes / 16 * 17}, options);
      char* const p = static_cast<char*>(d.data_ptr());
      (k ? s.codes_t : s.codes) = p;
      (k ? s.scales_t : s.scales) = p ? p + codes : nullptr;
      (of_t ? out[i].data_t : out[i].data) = d;
    }
    out[i].rows = turned ? s.cols : s.rows;
    out[i].cols = turned ? s.rows : s.cols;
  }
  check(library.quantize(sources.data(), n, stochastic, seed, stream_of(device)));
}

// mx_quantize(tensors, kinds, stochastic, seed) -> for each of a tuple of tensors (rows, cols, data,
// data_t); or the library's status.
PyObject* mx_quantize(PyObject*, PyObject* args) {
  PyObject* tuple;
  Buffer kinds;
  unsigned long long seed;
  int stochastic;
  if (!PyArg_ParseTuple(args, "O!y*pK", &PyTuple_Type, &tuple, &kinds.view, &stochastic, &seed))
    return nullptr;
  return answer([&]() -> PyObject* {
    const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
    if (n != kinds.view.len) throw Refused{PyExc_ValueError, "a kind for each tensor expected"};
    std::vector<const at::Tensor*> tensors(n);
    std::vector<Held> out(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const o = PyTuple_GET_ITEM(tuple, i);
      if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, "a tensor expected"};
      tensors[i] = &THPVariable_Unpack(o);
    }
    unlocked([&] {
      quantize(tensors.data(), static_cast<const char*>(kinds.view.buf), out.data(), n, stochastic, seed);
    });
    PyObject* const result = PyTuple_New(n);
    if (!result) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const each = Py_BuildValue("LLNN", (long long)out[i].rows, (long long)out[i].cols,
                                           THPVariable_Wrap(out[i].data), THPVariable_Wrap(out[i].data_t));
      if (!each) {
        Py_DECREF(result);
        return nullptr;
      }
      PyTuple_SET_ITEM(result, i, each);
    }
    return result;
  });
}

// The held form of rows x cols values: a uint8 tensor of the size that they take. (An empty one's
// address is not null.)
const char* held(const at::Tensor& t, int64_t rows, int64_t cols) {
  if (!t.defined() || !t.is_cuda() || t.scalar_type() != at::kByte || !t.is_contiguous() ||
      t.numel() != mx_codes(rows, cols) / 16 * 17)
    throw Refused{PyExc_ValueError, "held values of these sizes, on one device, expected"};
  static const char empty = 0;
  return t.numel() ? static_cast<const char*>(t.const_data_ptr()) : &empty;
}

const at::Tensor& tensor_of(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, "a tensor expected"};
  return THPVariable_Unpack(o);
}

at::ScalarType out_type(int dtype) { return dtype ? at::kFloat : at::kBFloat16; }

// mx_dequantize(data, rows, cols, dtype) -> a rows x cols tensor, or the status.
PyObject* mx_dequantize(PyObject*, PyObject* args) {
  PyObject* data;
  long long rows, cols;
  int dtype;
  if (!PyArg_ParseTuple(args, "OLLi", &data, &rows, &cols, &dtype)) return nullptr;
  return answer([&]() -> PyObject* {
    const at::Tensor& t = tensor_of(data);
    const char* const p = held(t, rows, cols);
    const at::Tensor out = unlocked([&] {
      const c10::DeviceGuard guard(t.device());
      at::Tensor out = at::empty({rows, cols}, at::TensorOptions().dtype(out_type(dtype)).device(t.device()));
      check(library.dequantize(p, p + mx_codes(rows, cols), rows, cols, out.data_ptr(), dtype,
                               stream_of(t.device())));
      return out;
    });
    return THPVariable_Wrap(out);
  });
}

// a b^T of held m x k and n x k values.
at::Tensor product(const at::Tensor& a, const at::Tensor& b, int64_t m, int64_t n, int64_t k, int dtype) {
  const char *const p = held(a, m, k), *const q = held(b, n, k);
  const at::Device device = a.device();
  if (b.device() != device) throw Refused{PyExc_ValueError, "held values of these sizes, on one device, expected"};
  const c10::DeviceGuard guard(device);
  const at::Tensor out = at::empty({m, n}, at::TensorOptions().dtype(out_type(dtype)).device(device));
  const size_t need = library.product_size(m, n, k);
  at::Tensor ws;
  if (need && need != SIZE_MAX)
    ws = at::empty({int64_t(need)}, at::TensorOptions().dtype(at::kByte).device(device));
  check(library.product(p, p + mx_codes(m, k), q, q + mx_codes(n, k), m, n, k, out.data_ptr(), dtype,
                        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? need : 0, stream_of(device)));
  return out;
}

// mx_matmul(a, b, m, n, k, dtype) -> an m x n tensor, or the status.
PyObject* mx_matmul(PyObject*, PyObject* args) {
  PyObject *a, *b;
  long long m, n, k;
  int dtype;
  if (!PyArg_ParseTuple(args, "OOLLLi", &a, &b, &m, &n, &k, &dtype)) return nullptr;
  return answer([&]() -> PyObject* {
    const at::Tensor &ta = tensor_of(a), &tb = tensor_of(b);
    return THPVariable_Wrap(unlocked([&] { return product(ta, tb, m, n, k, dtype); }));
  });
}

// A linear layer: y = Q(x) Q(w)^T; dx = Q(dy) Q(w^T)^T; dw = Q(dy^T) Q(x^T)^T. Between the passes it
// keeps x and w in 4 bits. (As a Python function its two passes take 101 us of host time, 49 of them
// PyTorch's own for any such function.)
struct LinearCall {
  at::Tensor rows, cols;                         // the weight as held, or undefined
  bool need_x, need_w, stochastic;
  int64_t seed;
};

// t, or a copy of it in rows of its last dimension where it does not lie as quantize takes it.
at::Tensor rows_laid(const at::Tensor& t) {
  MxSource s;
  bool transposed;
  return !t.is_neg() && rows_of(t, s, transposed) ? t : t.resolve_neg().contiguous();
}

class Linear : public torch::autograd::Function<Linear> {
 public:
  static at::Tensor forward(torch::autograd::AutogradContext* ctx, const at::Tensor& x, const at::Tensor& w,
                            const LinearCall& call) {
    const int64_t o = w.size(0);
    const bool own = !call.rows.defined();
    const at::Tensor xr = rows_laid(x), wr = own ? rows_laid(w) : w;
    Held h[2];
    const at::Tensor* const tensors[2] = {&xr, &wr};
    const char kinds[2] = {char(call.need_w ? 3 : 1), char(call.need_x ? 3 : 1)};
    quantize(tensors, kinds, h, own ? 2 : 1, false, 0);
    const Held& hx = h[0];
    const at::Tensor y = product(hx.data, own ? h[1].data : call.rows, hx.rows, o, hx.cols, dtype_code(x));
    ctx->save_for_backward({call.need_w ? hx.data_t : at::Tensor(),
                            !call.need_x ? at::Tensor() : own ? h[1].data_t : call.cols});
    ctx->saved_data["sizes"] = std::vector<int64_t>{hx.rows, hx.cols, o};
    ctx->saved_data["shape"] = x.sizes().vec();
    ctx->saved_data["how"] = std::vector<int64_t>{dtype_code(x), dtype_code(w), call.stochastic, call.seed};
    if (x.dim() == 2) return y;
    std::vector<int64_t> shape = x.sizes().vec();
    shape.back() = o;
    return at::_unsafe_view(y, shape);           // (autograd refuses to change a view made in here)
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    try {
      return both(ctx, grads[0]);
    } catch (const Refused& e) {
      throw std::runtime_error(e.text);
    } catch (const Failed&) {
      throw std::runtime_error(library.last_error());
    }
  }

 private:
  static torch::autograd::variable_list both(torch::autograd::AutogradContext* ctx, const at::Tensor& grad) {
    const auto saved = ctx->get_saved_variables();
    const auto sizes = ctx->saved_data["sizes"].toIntVector();
    const auto how = ctx->saved_data["how"].toIntVector();
    const int64_t t = sizes[0], i = sizes[1], o = sizes[2];
    const bool need_x = saved[1].defined() && ctx->needs_input_grad(0);
    const bool need_w = saved[0].defined() && ctx->needs_input_grad(1);
    at::Tensor dx, dw;
    if (need_x || need_w) {
      const at::AutoGradMode no_grad(false);
      // (an expanded gradient, of a sum say, has no memory of its own for each value)
      const at::Tensor dy = grad.resolve_neg().contiguous().view({t, o});
      const at::Tensor* const tensor = &dy;
      const char kind = char((need_x ? 1 : 0) | (need_w ? 2 : 0));
      Held h;
      quantize(&tensor, &kind, &h, 1, how[2], uint64_t(how[3]));
      if (need_x)
        dx = at::_unsafe_view(product(h.data, saved[1], t, i, o, int(how[0])),
                              ctx->saved_data["shape"].toIntVector());
      if (need_w) dw = product(h.data_t, saved[0], o, i, t, int(how[1]));
    }
    if (at::GradMode::is_enabled()) {
      // results of a pass that is itself recorded: what would differentiate them raises. dx is a function of
      // the weight, dw of x, also where dy is a constant
      auto guard = [](at::Tensor& v) {
        if (!v.defined()) return;
        const auto error = std::make_shared<torch::autograd::DelayedError>("mx4_linear is differentiable once", 1);
        v.requires_grad_(true);
        v = (*error)({v})[0];
      };
      if (grad.requires_grad() || saved[0].defined()) guard(dx);
      if (grad.requires_grad() || saved[1].defined()) guard(dw);
    }
    return {dx, dw, at::Tensor()};
  }
};

// mx_linear(x, weight, rows, cols, stochastic, seed) -> y, or the status. rows, cols: the weight and its
// transpose as held, or None.
PyObject* mx_linear(PyObject*, PyObject* args) {
  PyObject *x, *w, *rows, *cols;
  int stochastic;
  long long seed;
  if (!PyArg_ParseTuple(args, "OOOOpL", &x, &w, &rows, &cols, &stochastic, &seed)) return nullptr;
  return answer([&]() -> PyObject* {
    const at::Tensor &tx = tensor_of(x), &tw = tensor_of(w);
    const bool grad = at::GradMode::is_enabled();
    LinearCall call{rows == Py_None ? at::Tensor() : tensor_of(rows),
                    cols == Py_None ? at::Tensor() : tensor_of(cols),
                    grad && tx.requires_grad(), grad && tw.requires_grad(), bool(stochastic), seed};
    return THPVariable_Wrap(unlocked([&] { return Linear::apply(tx, tw, call); }));
  });
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

// A new tensor of x's shape, dense, its dimensions in x's order of strides.
at::Tensor dense_like(const at::Tensor& x, at::ScalarType type) {
  const int64_t d = x.dim();
  std::vector<int64_t> order(d), strides(d);
  for (int64_t i = 0; i < d; ++i) order[i] = i;
  auto far = [&](int64_t i) {                    // (a dimension without strides goes outside)
    return x.size(i) > 1 && x.stride(i) == 0 ? INT64_MAX : x.stride(i);
  };
  std::stable_sort(order.begin(), order.end(), [&](int64_t a, int64_t b) { return far(a) > far(b); });
  int64_t step = 1;
  for (int64_t i = d; i-- > 0;) {
    strides[order[i]] = step;
    step *= std::max<int64_t>(x.size(order[i]), 1);
  }
  return at::empty_strided(x.sizes(), strides, at::TensorOptions().dtype(type).device(x.device()));
}

// muon_orthogonalize of x into out, tensors of equal sizes, dtypes and devices.
void orthogonalize_into(const at::Tensor& x, const at::Tensor& out, const void* cfg) {
  const int64_t d = x.dim();
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
    if (groups == 2) throw Refused{PyExc_ValueError, "leading dimensions of more than two strides"};
    sides[groups] = n;
    si[groups] = x.stride(i);
    so[groups] = out.stride(i);
    ++groups;
  }
  for (int j = 0; j < 2; ++j) {                  // group 0 is the inner one
    k.side[1 - j] = sides[j];
    k.in_stride[1 - j] = si[j];
    k.out_stride[1 - j] = so[j];
    k.side[2 + j] = x.size(d - 2 + j);
    k.in_stride[2 + j] = x.stride(d - 2 + j);
    k.out_stride[2 + j] = out.stride(d - 2 + j);
  }
  const size_t need = library.stacked_size(k.side[0], k.side[1], k.side[2], k.side[3]);
  at::Tensor ws;
  if (need && need != SIZE_MAX)
    ws = at::empty({int64_t(need)}, at::TensorOptions().dtype(at::kByte).device(x.device()));
  check(library.stacked(&k, cfg, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? need : 0,
                        stream_of(x.device())));
}

// orthogonalize(x, out, cfg) -> out (a new tensor in x's order of strides where it is None), or the
// status. x: at least 2-D, its leading dimensions two strides at most.
PyObject* orthogonalize(PyObject*, PyObject* args) {
  PyObject *xo, *oo;
  Buffer cfg;
  if (!PyArg_ParseTuple(args, "OOy*", &xo, &oo, &cfg.view)) return nullptr;
  return answer([&]() -> PyObject* {
    const at::Tensor& x = tensor_of(xo);
    if (!x.is_cuda() || x.layout() != at::kStrided || x.is_neg())
      throw Refused{PyExc_ValueError, "a CUDA tensor whose memory holds its values expected"};
    if (dtype_code(x) != 0 && dtype_code(x) != 1)
      throw Refused{PyExc_TypeError, "unsupported dtype: the library takes bfloat16 or float32"};
    if (x.dim() < 2) throw Refused{PyExc_ValueError, "a matrix or a stack of them expected"};
    const c10::DeviceGuard guard(x.device());
    at::Tensor out;
    if (oo == Py_None) {
      out = dense_like(x, x.scalar_type());
    } else {
      out = tensor_of(oo);
      if (out.device() != x.device() || out.scalar_type() != x.scalar_type() ||
          out.sizes() != x.sizes() || out.layout() != at::kStrided || out.is_neg())
        throw Refused{PyExc_ValueError, "out must be a tensor of x's shape, dtype and device"};
    }
    if (x._fw_grad(0).defined() || out._fw_grad(0).defined())
      throw Refused{PyExc_ValueError, "orthogonalize has no forward-mode derivative: call it on primal values"};
    const int passes = library.passes(cfg.view.buf);
    check(std::min(passes, 0));
    unlocked([&] {
      if (passes > 1 && dtype_code(x) == 0) {    // bf16 values are held in fp32 between passes
        const at::AutoGradMode no_grad(false);
        at::Tensor wide = dense_like(x, at::kFloat);
        wide.copy_(x);
        orthogonalize_into(wide, wide, cfg.view.buf);
        out.copy_(wide);
      } else {
        orthogonalize_into(x, out, cfg.view.buf);
      }
    });
    // (what autograd saved of the result's tensor before is not its value any more)
    if (oo != Py_None && !out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
    return THPVariable_Wrap(out);
  });
}

PyMethodDef methods[] = {
    {"orthogonalize", orthogonalize, METH_VARARGS, "muon_orthogonalize of a stack."},
    {"mx_quantize", mx_quantize, METH_VARARGS, "muon_mx_quantize of tensors into new ones."},
    {"mx_dequantize", mx_dequantize, METH_VARARGS, "muon_mx_dequantize into a new tensor."},
    {"mx_matmul", mx_matmul, METH_VARARGS, "muon_mx_matmul into a new tensor."},
    {"mx_linear", mx_linear, METH_VARARGS, "A linear layer of microscaled 4-bit products."},
    {"bind", bind, METH_VARARGS, "The addresses of the library's functions."},
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
