// The binding's checks of tensor arguments (Python module _args): a call of
// microseconds of GPU work has up to fifteen tensors, and looking at one from
// Python takes 0.33 us (five attribute reads), here 0.03.
//
//   built_for                       the torch whose objects this reads
//   use(error)                      the exception that refusals raise
//   addresses(device, what, t, dtype, shape, ...)  four arguments a tensor; the
//       addresses of contiguous tensors of these types and shapes on that CUDA
//       device.  dtype None: any dtype, the last dimension contiguous; address and
//       the two other strides of [T][H][D].  dtype and shape None: any contiguous
//       tensor; address and bytes.  t None: 0 where `what` ends in '?', else
//       refused.
#include <c10/core/ScalarType.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

namespace {

PyObject* g_error = nullptr;

std::string list_of(c10::IntArrayRef x) {
  std::string s = "[";
  for (size_t i = 0; i < x.size(); ++i) s += (i ? ", " : "") + std::to_string(x[i]);
  return s + "]";
}
std::string text(PyObject* o) {
  PyObject* s = PyObject_Str(o);
  const char* c = s ? PyUnicode_AsUTF8(s) : nullptr;
  const std::string r = c ? c : "?";
  Py_XDECREF(s);
  if (!c) PyErr_Clear();
  return r;
}
PyObject* refuse(const std::string& message) {
  PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, message.c_str());
  return nullptr;
}
bool same_shape(c10::IntArrayRef have, PyObject* want) {
  if (!PyTuple_Check(want) || PyTuple_GET_SIZE(want) != (Py_ssize_t)have.size()) return false;
  for (size_t i = 0; i < have.size(); ++i) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(want, i));
    if (n != have[i]) {
      PyErr_Clear();
      return false;
    }
  }
  return true;
}

PyObject* use(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

PyObject* checked_addresses(PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t MOST = 64;
  long long out[MOST];
  Py_ssize_t m = 0;
  if (n % 4 != 1) return refuse("a device and four arguments a tensor");
  const long device = PyLong_AsLong(a[0]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  auto elsewhere = [&](PyObject* what, const at::Tensor& x) {
    return refuse(text(what) + " is on " + x.device().str() + ", the call on cuda:" + std::to_string(device));
  };
  for (Py_ssize_t i = 1; i < n; i += 4) {
    if (m + 3 > MOST) return refuse("too many tensors");
    PyObject *what = a[i], *t = a[i + 1], *dtype = a[i + 2], *shape = a[i + 3];
    if (t == Py_None) {
      const std::string name = text(what);
      if (name.empty() || name.back() != '?') return refuse(name + " is missing");
      out[m++] = 0;
      continue;
    }
    if (!THPVariable_Check(t)) return refuse(text(what) + " must be a tensor");
    const at::Tensor& x = THPVariable_Unpack(t);
    if (dtype == Py_None && shape != Py_None) {
      if (!same_shape(x.sizes(), shape) || x.dim() != 3 || x.stride(2) != 1)
        return refuse(text(what) + " must be " + text(shape) + " with a contiguous last dimension, not " + list_of(x.sizes()) +
                      " with strides " + list_of(x.strides()));
      if (!x.is_cuda()) return refuse(text(what) + " must be a CUDA tensor");
      if (x.device().index() != device) return elsewhere(what, x);
      out[m++] = (long long)(uintptr_t)x.data_ptr();
      out[m++] = x.stride(0);
      out[m++] = x.stride(1);
      continue;
    }
    if (dtype == Py_None) {
      if (!x.is_cuda() || !x.is_contiguous()) return refuse(text(what) + " must be a contiguous CUDA tensor");
      if (x.device().index() != device) return elsewhere(what, x);
      out[m++] = (long long)(uintptr_t)x.data_ptr();
      out[m++] = (long long)x.nbytes();
      continue;
    }
    if (!THPDtype_Check(dtype)) return refuse("a dtype is expected for " + text(what));
    if (x.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type || !same_shape(x.sizes(), shape))
      return refuse(text(what) + " must be " + text(dtype) + " " + text(shape) + ", not " + c10::toString(x.scalar_type()) +
                    " " + list_of(x.sizes()));
    if (!x.is_cuda() || !x.is_contiguous()) return refuse(text(what) + " must be a contiguous CUDA tensor");
    if (x.device().index() != device) return elsewhere(what, x);
    out[m++] = (long long)(uintptr_t)x.data_ptr();
  }
  PyObject* r = PyTuple_New(m);
  if (!r) return nullptr;
  for (Py_ssize_t i = 0; i < m; ++i) {
    PyObject* v = PyLong_FromLongLong(out[i]);
    if (!v) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, v);
  }
  return r;
}

// torch throws where a kind of tensor has no sizes, strides or address.
PyObject* addresses(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return checked_addresses(a, n);
  } catch (const c10::Error& e) {
    return refuse(std::string("not a plain tensor: ") + e.what_without_backtrace());
  } catch (const std::exception& e) {
    return refuse(e.what());
  } catch (...) {
    return refuse("an unknown exception in the checks of tensors");
  }
}

PyMethodDef methods[] = {
    {"use", use, METH_O, "The exception that refusals raise."},
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(addresses)), METH_FASTCALL,
     "Checked addresses (and strides) of tensors."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", "Checks of tensor arguments.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__args() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", SPEC_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
