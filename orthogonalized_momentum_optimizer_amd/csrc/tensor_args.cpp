// Checks a list of tensors against a plan and collects their addresses, in one pass of native
// code. The steps over many small tensors take a few microseconds on the GPU, less than the same
// checks take from Python (122 tensors: 45 us from Python, 1 us here).
//
// Host code only: built with the C++ compiler against PyTorch's headers.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

// muon_dtype of a tensor, -1 if the library has none for it
int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return 0;
    case at::kFloat: return 1;
    default: return -1;
  }
}

bool fits(const at::Tensor& t, int64_t numel, int dtype, long device) {
  return t.is_cuda() && t.get_device() == device && t.numel() == numel &&
         dtype_code(t) == dtype && t.is_contiguous();
}

// addresses(tensors, numels, dtypes, device, out) -> -1, or the index of the first entry that is
// neither None (address 0) nor a contiguous tensor of its size and dtype on the device.
// tensors: a list or tuple; numels, dtypes, out: buffers of int64, int32 and uint64 of its length.
PyObject* addresses(PyObject*, PyObject* args) {
  PyObject* tensors;
  Py_buffer numels, dtypes, out;
  long device;
  if (!PyArg_ParseTuple(args, "Oy*y*lw*", &tensors, &numels, &dtypes, &device, &out)) return nullptr;
  PyObject* result = nullptr;
  PyObject* fast = PySequence_Fast(tensors, "a list or tuple of tensors expected");
  if (fast) {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    if (numels.len != n * 8 || dtypes.len != n * 4 || out.len != n * 8) {
      PyErr_SetString(PyExc_ValueError, "buffers and tensors differ in length");
    } else {
      PyObject** const items = PySequence_Fast_ITEMS(fast);
      const int64_t* const numel = static_cast<const int64_t*>(numels.buf);
      const int32_t* const dtype = static_cast<const int32_t*>(dtypes.buf);
      uint64_t* const to = static_cast<uint64_t*>(out.buf);
      Py_ssize_t bad = -1;
      for (Py_ssize_t i = 0; i < n && bad < 0; ++i) {
        if (items[i] == Py_None) {
          to[i] = 0;
          continue;
        }
        try {
          if (THPVariable_Check(items[i]) &&
              fits(THPVariable_Unpack(items[i]), numel[i], dtype[i], device))
            to[i] = reinterpret_cast<uint64_t>(THPVariable_Unpack(items[i]).const_data_ptr());
          else
            bad = i;
        } catch (...) {                          // a tensor without storage
          bad = i;
        }
      }
      result = PyLong_FromSsize_t(bad);
    }
    Py_DECREF(fast);
  }
  PyBuffer_Release(&numels);
  PyBuffer_Release(&dtypes);
  PyBuffer_Release(&out);
  return result;
}

PyMethodDef methods[] = {
    {"addresses", addresses, METH_VARARGS, "Addresses of the tensors of a plan's layout."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
