// Lists of tensors as the library's host arrays: addresses, sizes and types of
// a thousand tensors and more, checked, in one call from Python (by the
// interpreter each property of each tensor costs about 0.1 us, for 1500 tensors
// several times what the kernels take).
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

#include <stdexcept>
#include <string>

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// One tensor of `name`: its type code (0 float32, 1 bfloat16).
int32_t check(const at::Tensor &t, int64_t dev, const char *name) {
  const auto type = t.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    throw Refused(std::string(name) + ": torch.float32 or torch.bfloat16 expected, got " + c10::toString(type));
  if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev)
    throw Refused(std::string(name) + ": dense tensors on device " + std::to_string(dev) + " expected, got one on " +
                  t.device().str());
  if (t.numel() && !t.is_non_overlapping_and_dense())
    throw Refused(std::string(name) + ": tensors without gaps expected, got strides " + shape_of(t.strides()) + " of " +
                  shape_of(t.sizes()));
  return type == at::kFloat ? 0 : 1;
}

const at::Tensor &tensor(PyObject *list, Py_ssize_t i, const char *name) {
  PyObject *o = PyList_GET_ITEM(list, i);
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": tensors expected");
  return THPVariable_Unpack(o);
}

// pack(grads, out or None, device) -> (arrays, address of in, out, numel, dtype, odtype).
// The addresses hold as long as `arrays` lives.
PyObject *pack(PyObject *, PyObject *args) {
  PyObject *grads, *out;
  long long dev;
  if (!PyArg_ParseTuple(args, "O!OL", &PyList_Type, &grads, &out, &dev)) return nullptr;
  const bool other = out != Py_None;
  if (other && !PyList_Check(out)) {
    PyErr_SetString(PyExc_TypeError, "out: a list expected");
    return nullptr;
  }
  const Py_ssize_t n = PyList_GET_SIZE(grads);
  PyObject *blob = PyBytes_FromStringAndSize(nullptr, n * (3 * 8 + 2 * 4) + 8);
  if (!blob) return nullptr;
  const uintptr_t base = ((uintptr_t)PyBytes_AS_STRING(blob) + 7) & ~(uintptr_t)7;
  auto *in_at = (uint64_t *)base, *out_at = in_at + n;
  auto *numel = (int64_t *)(out_at + n);
  auto *type = (int32_t *)(numel + n), *otype = type + n;
  try {
    if (other && PyList_GET_SIZE(out) != n)
      throw Refused("out: " + std::to_string(n) + " tensors expected, got " + std::to_string(PyList_GET_SIZE(out)));
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor &g = tensor(grads, i, "grads");
      type[i] = otype[i] = check(g, dev, "grads");
      numel[i] = g.numel();
      in_at[i] = out_at[i] = (uint64_t)g.data_ptr();
      if (!other) continue;
      const at::Tensor &o = tensor(out, i, "out");
      otype[i] = check(o, dev, "out");
      out_at[i] = (uint64_t)o.data_ptr();
      // Elements in the same order: both in that of their indices, or with equal strides.
      if (o.numel() != g.numel() ||
          (!(g.is_contiguous() && o.is_contiguous()) && (g.sizes() != o.sizes() || g.strides() != o.strides())))
        throw Refused("out: " + shape_of(g.sizes()) + " with strides " + shape_of(g.strides()) + " expected, got " +
                      shape_of(o.sizes()) + " with " + shape_of(o.strides()));
    }
  } catch (const Refused &e) {
    Py_DECREF(blob);
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  } catch (const std::exception &e) {
    Py_DECREF(blob);
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return Py_BuildValue("(NKKKKK)", blob, (unsigned long long)(uintptr_t)in_at, (unsigned long long)(uintptr_t)out_at,
                       (unsigned long long)(uintptr_t)numel, (unsigned long long)(uintptr_t)type,
                       (unsigned long long)(uintptr_t)otype);
}

PyMethodDef methods[] = {{"pack", pack, METH_VARARGS, "Addresses, sizes and types of lists of tensors."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_list", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_list() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
