// _tensors.cpp -- the checks of a call's tensors in one pass.
//
// A decode step's calls take up to a dozen tensors each.  Asking every one for
// its device, type, layout, shape and address through Python cost 5 to 11 us a
// call, more than the launch (2.5 us) and for small steps more than the
// kernels; here it takes 1.  `fit` only looks: what does not fit is None, and
// the Python module says what it was.  It has the same function in Python for
// where this was not built, or was built for another torch (torch_version),
// whose tensors may be laid out differently.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kMaxOut = 64;

// One letter a dimension: the value it had where it came first, the order in
// which the letters came.
struct Dims {
  int64_t value[26];
  int order[26], n = 0;
  uint32_t seen = 0, bound = 0;
  void name(char c) {  // (also of tensors that are not there)
    const int i = c - 'A';
    if (!(seen >> i & 1u)) {
      seen |= 1u << i;
      order[n++] = i;
      value[i] = -1;
    }
  }
  bool match(char c, int64_t size) {
    const int i = c - 'A';
    name(c);
    if (bound >> i & 1u) return value[i] == size;
    bound |= 1u << i;
    value[i] = size;
    return size >= 0;
  }
};

PyObject* look(PyObject* const* a, Py_ssize_t n_args) {
  Py_ssize_t len = 0;
  const char* s = n_args > 0 ? PyUnicode_AsUTF8AndSize(a[0], &len) : nullptr;
  if (s == nullptr) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "fit takes a layout and tensors");
    return nullptr;
  }
  const char* const end = s + len;
  Dims dims;
  c10::IntArrayRef any;  // what @ stands for
  bool has_any = false;
  int device = -1, n_out = 0;
  int64_t out[kMaxOut];
  bool none[kMaxOut];
  auto put = [&](int64_t v, bool is_none) {
    out[n_out] = v;
    none[n_out++] = is_none;
  };
  for (Py_ssize_t k = 1;; ++k) {
    while (s < end && *s == ' ') ++s;
    if (s == end) {
      if (k == n_args) break;
      PyErr_SetString(PyExc_TypeError, "fit: more tensors than the layout has");
      return nullptr;
    }
    if (k == n_args || n_out + 2 > kMaxOut) {
      PyErr_SetString(PyExc_TypeError, "fit: fewer tensors than the layout has");
      return nullptr;
    }
    const bool optional = *s == '?';
    if (optional) ++s;
    const char type = *s++;
    if (optional && a[k] == Py_None) {
      for (; s < end && *s != ' '; ++s)
        if (*s >= 'A' && *s <= 'Z') dims.name(*s);
      put(0, true);
      if (type == 'w') put(0, false);
      continue;
    }
    if (!THPVariable_Check(a[k])) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(a[k]);
    if (!t.is_cuda() || (k > 1 && t.get_device() != device)) Py_RETURN_NONE;
    device = (int)t.get_device();
    const auto want = type == 'u' ? at::kByte : type == 'i' ? at::kInt : type == 'f' ? at::kFloat : at::kBFloat16;
    if (type != 'w' && t.scalar_type() != want) Py_RETURN_NONE;
    const c10::IntArrayRef sizes = t.sizes();
    size_t i = 0;
    bool whole = false, first_any = false;
    for (; s < end && *s != ' '; ++s) {
      if (*s == '@') {
        if (!has_any) {
          any = sizes;
          has_any = first_any = true;
          i = sizes.size();
        } else {
          for (int64_t d : any)
            if (i == sizes.size() || sizes[i++] != d) Py_RETURN_NONE;
        }
        continue;
      }
      if (i == sizes.size()) Py_RETURN_NONE;
      const bool more = s + 1 < end && s[1] == '+';
      if (!dims.match(*s, sizes[i++] - (more ? 1 : 0))) Py_RETURN_NONE;
      if (more) ++s;
    }
    whole = type == 'w' || i == sizes.size();
    if (!whole) Py_RETURN_NONE;
    if (type == 'q') {  // rows of [heads][head_dim], any distance apart
      const c10::IntArrayRef st = t.strides();
      if (sizes.size() != 3 || !(st[2] == 1 || sizes[2] == 1) || !(st[1] == sizes[2] || sizes[1] == 1)) Py_RETURN_NONE;
      put((int64_t)(intptr_t)t.data_ptr(), false);
      put(sizes[0] > 1 ? st[0] : sizes[1] * sizes[2], false);
      continue;
    }
    if (!t.is_contiguous()) Py_RETURN_NONE;
    put((int64_t)(intptr_t)t.data_ptr(), false);
    if (type == 'w') put((int64_t)t.nbytes(), false);
    else if (first_any) put(t.numel(), false);
  }
  PyObject* r = PyTuple_New(1 + dims.n + n_out);
  if (r == nullptr) return nullptr;
  Py_ssize_t at = 0;
  auto set = [&](PyObject* x) { PyTuple_SET_ITEM(r, at++, x); };
  set(PyLong_FromLong(device));
  for (int i = 0; i < dims.n; ++i) set(PyLong_FromLongLong(dims.value[dims.order[i]]));
  for (int i = 0; i < n_out; ++i) {
    if (none[i]) set(Py_NewRef(Py_None));
    else set(PyLong_FromLongLong(out[i]));
  }
  if (PyErr_Occurred()) {
    Py_DECREF(r);
    return nullptr;
  }
  return r;
}

// fit(spec, tensors...): see _fit_py in the Python module.  Tensors without
// sizes, strides or an address (sparse ones, those inside vmap) throw when they
// are asked for them.
PyObject* fit(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  try {
    return look(a, n_args);
  } catch (const c10::Error& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"fit", (PyCFunction)(void (*)(void))fit, METH_FASTCALL, "Sizes and addresses of tensors that fit a layout, else None."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "Checks of a call's tensors in one pass.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", QSA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
