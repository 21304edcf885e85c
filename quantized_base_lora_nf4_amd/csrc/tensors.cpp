// What the Python binding reads of every tensor in a list, in one call: at
// hundreds of tensors per optimizer step the attributes, read one by one from
// Python, take longer than the step's kernels.  Whatever is not the ordinary
// case is left to the Python code, which names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <exception>
#include <vector>

#include <torch/csrc/autograd/python_variable.h>

namespace {

// describe(tensors, ptrs, sizes, types, bf16, f32) -> int
//
// tensors: a list; ptrs, sizes, types: addresses of as many uint64, int64 and
// int32, which take each tensor's address, number of elements and type (the
// numbers bf16 and f32).  Returns the index of the GPU that all are on; -1 if
// one of them is not a contiguous bfloat16 or float32 tensor of the first one's
// GPU.
PyObject* describe(PyObject*, PyObject* args) {
  PyObject* list;
  unsigned long long ptrs, sizes, types;
  int bf16, f32;
  if (!PyArg_ParseTuple(args, "O!KKKii", &PyList_Type, &list, &ptrs, &sizes, &types, &bf16, &f32))
    return nullptr;
  long device = -1;
  try {
    const Py_ssize_t n = PyList_GET_SIZE(list);
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const o = PyList_GET_ITEM(list, i);
      if (!THPVariable_Check(o)) return PyLong_FromLong(-1);
      const at::Tensor& t = THPVariable_Unpack(o);
      const c10::ScalarType ty = t.scalar_type();
      if (!t.is_cuda() || t.layout() != c10::kStrided ||
          (ty != c10::ScalarType::BFloat16 && ty != c10::ScalarType::Float) || !t.is_contiguous())
        return PyLong_FromLong(-1);
      if (i == 0) device = t.get_device();
      if (t.get_device() != device) return PyLong_FromLong(-1);
      reinterpret_cast<uint64_t*>(ptrs)[i] = reinterpret_cast<uint64_t>(t.data_ptr());
      reinterpret_cast<int64_t*>(sizes)[i] = t.numel();
      reinterpret_cast<int32_t*>(types)[i] = ty == c10::ScalarType::Float ? f32 : bf16;
    }
  } catch (...) {
    return PyLong_FromLong(-1);
  }
  return PyLong_FromLong(device);
}

// same_shapes(a, b) -> bool: two lists of tensors, as many with the same shapes.
PyObject* same_shapes(PyObject*, PyObject* args) {
  PyObject *a, *b;
  if (!PyArg_ParseTuple(args, "O!O!", &PyList_Type, &a, &PyList_Type, &b)) return nullptr;
  try {
    const Py_ssize_t n = PyList_GET_SIZE(a);
    if (PyList_GET_SIZE(b) != n) Py_RETURN_FALSE;
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject *const x = PyList_GET_ITEM(a, i), *const y = PyList_GET_ITEM(b, i);
      if (!THPVariable_Check(x) || !THPVariable_Check(y) ||
          THPVariable_Unpack(x).sizes() != THPVariable_Unpack(y).sizes())
        Py_RETURN_FALSE;
    }
  } catch (...) {
    Py_RETURN_FALSE;
  }
  Py_RETURN_TRUE;
}

bool type_fits(char kind, c10::ScalarType t) {
  switch (kind) {
    case 's':
      return t == c10::ScalarType::BFloat16 || t == c10::ScalarType::Short ||
             t == c10::ScalarType::UInt16;
    case 'f':
      return t == c10::ScalarType::Float;
    case 'i':
      return t == c10::ScalarType::Int;
    case 'b':
      return t == c10::ScalarType::Byte;
    case 'c':
      return t == c10::ScalarType::Char;
    default:
      return false;
  }
}

// fits(device, kinds, tensors, shapes) -> bool: each of the tuple `tensors` is a
// contiguous tensor on GPU `device`, of the type that its letter in `kinds`
// names (s: 16 bits as the layer takes them, f: float32, i: int32, b: uint8, c:
// int8) and of the shape in the tuple `shapes`.
PyObject* fits(PyObject*, PyObject* args) {
  long device;
  const char* kinds;
  Py_ssize_t n;
  PyObject *list, *shapes;
  if (!PyArg_ParseTuple(args, "ls#O!O!", &device, &kinds, &n, &PyTuple_Type, &list, &PyTuple_Type,
                        &shapes))
    return nullptr;
  if (PyTuple_GET_SIZE(list) != n || PyTuple_GET_SIZE(shapes) != n) Py_RETURN_FALSE;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject *const o = PyTuple_GET_ITEM(list, i), *const shape = PyTuple_GET_ITEM(shapes, i);
      if (!THPVariable_Check(o) || !PyTuple_Check(shape)) Py_RETURN_FALSE;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != device ||
          !type_fits(kinds[i], t.scalar_type()) || !t.is_contiguous() ||
          t.dim() != PyTuple_GET_SIZE(shape))
        Py_RETURN_FALSE;
      for (int64_t d = 0; d < t.dim(); ++d) {
        const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
        if (want == -1 && PyErr_Occurred()) return nullptr;
        if (t.size(d) != want) Py_RETURN_FALSE;
      }
    }
  } catch (...) {
    Py_RETURN_FALSE;
  }
  Py_RETURN_TRUE;
}

// distinct(ptrs, n) -> bool: n addresses, no two alike.
PyObject* distinct(PyObject*, PyObject* args) {
  unsigned long long ptrs;
  Py_ssize_t n;
  if (!PyArg_ParseTuple(args, "Kn", &ptrs, &n)) return nullptr;
  const uint64_t* const p = reinterpret_cast<const uint64_t*>(ptrs);
  Py_ssize_t i = 1;
  while (i < n && p[i - 1] < p[i]) ++i;
  if (i >= n) Py_RETURN_TRUE;  // in order already
  try {
    std::vector<uint64_t> s(p, p + n);
    std::sort(s.begin(), s.end());
    if (std::adjacent_find(s.begin(), s.end()) == s.end()) Py_RETURN_TRUE;
  } catch (...) {
  }
  Py_RETURN_FALSE;
}

// written(tensors): each tensor in a list or tuple (None entries are passed
// over) counts a new version, as after torch's own operations in place: a
// backward pass that saved it before raises.  Inference tensors have none.
PyObject* written(PyObject*, PyObject* arg) {
  PyObject* const seq = PySequence_Fast(arg, "expected a list or tuple of tensors");
  if (!seq) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  PyObject* const* const items = PySequence_Fast_ITEMS(seq);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (items[i] == Py_None) continue;
    if (!THPVariable_Check(items[i])) {
      Py_DECREF(seq);
      PyErr_SetString(PyExc_TypeError, "expected tensors");
      return nullptr;
    }
    try {
      const at::Tensor& t = THPVariable_Unpack(items[i]);
      if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    } catch (const std::exception& e) {
      Py_DECREF(seq);
      PyErr_SetString(PyExc_RuntimeError, e.what());
      return nullptr;
    }
  }
  Py_DECREF(seq);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"describe", describe, METH_VARARGS, nullptr},
                         {"same_shapes", same_shapes, METH_VARARGS, nullptr},
                         {"fits", fits, METH_VARARGS, nullptr},
                         {"distinct", distinct, METH_VARARGS, nullptr},
                         {"written", written, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
