// dkv_python.cpp -- CPython calls of the entry points a serving step makes.
//
// A step's small calls are bound by the host: converting 14 to 22 arguments
// through ctypes costs 4 to 6 us of interpreter time, more than their kernels
// run.  Here an argument is read straight from its object: None is a null
// pointer, a whole number itself, anything else (a tensor) what its data_ptr()
// returns.  The library is opened by the path that the package gives, so both
// always talk to the same build.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "dkv.h"

namespace {

PyObject* g_data_ptr = nullptr;   // the interned method name

struct Entries {
  decltype(&dkv_extend_tables) extend_tables = nullptr;
  decltype(&dkv_store_kv) store_kv = nullptr;
  decltype(&dkv_attn_chunk) attn_chunk = nullptr;
  decltype(&dkv_attn_decode_window) attn_decode_window = nullptr;
} g_entries;

template <class T>
bool read(PyObject* o, T& out) {
  if constexpr (std::is_pointer_v<T>) {
    if (o == Py_None) {
      out = nullptr;
      return true;
    }
    PyObject* p = o;
    if (PyLong_Check(o)) Py_INCREF(p);
    else if (!(p = PyObject_CallMethodNoArgs(o, g_data_ptr))) return false;
    out = reinterpret_cast<T>(PyLong_AsVoidPtr(p));
    Py_DECREF(p);
    return !PyErr_Occurred();
  } else {
    PyObject* p = PyNumber_Index(o);
    if (!p) return false;
    const long long v = PyLong_AsLongLong(p);
    Py_DECREF(p);
    if (v == -1 && PyErr_Occurred()) return false;
    out = static_cast<T>(v);
    if (static_cast<long long>(out) != v) {
      PyErr_SetString(PyExc_OverflowError, "argument does not fit its C type");
      return false;
    }
    return true;
  }
}

template <class... A, size_t... I>
PyObject* invoke(int (*fn)(A...), PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
  if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
    PyErr_Format(PyExc_TypeError, "%zu arguments are needed, %zd were given", sizeof...(A), n);
    return nullptr;
  }
  std::tuple<A...> v;
  if (!(read(args[I], std::get<I>(v)) && ...)) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(std::get<I>(v)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

template <class F>
PyObject* call(F fn, PyObject* const* args, Py_ssize_t n);
template <class... A>
PyObject* call(int (*fn)(A...), PyObject* const* args, Py_ssize_t n) {
  if (!fn) {
    PyErr_SetString(PyExc_RuntimeError, "load() has not been called");
    return nullptr;
  }
  return invoke(fn, args, n, std::index_sequence_for<A...>{});
}

PyObject* extend_tables(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(g_entries.extend_tables, a, n); }
PyObject* store_kv(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(g_entries.store_kv, a, n); }
PyObject* attn_chunk(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(g_entries.attn_chunk, a, n); }
PyObject* attn_decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(g_entries.attn_decode_window, a, n);
}

template <class F>
bool find(void* lib, const char* name, F& out) {
  out = reinterpret_cast<F>(dlsym(lib, name));
  if (!out) PyErr_Format(PyExc_ImportError, "the library has no %s", name);
  return out != nullptr;
}

// load(path): the entry points of the library at `path`.
PyObject* load(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_Format(PyExc_ImportError, "%s", dlerror());
    return nullptr;
  }
  if (!find(lib, "dkv_extend_tables", g_entries.extend_tables) || !find(lib, "dkv_store_kv", g_entries.store_kv) ||
      !find(lib, "dkv_attn_chunk", g_entries.attn_chunk) ||
      !find(lib, "dkv_attn_decode_window", g_entries.attn_decode_window))
    return nullptr;
  Py_RETURN_NONE;
}

#define DKV_FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DKV_FAST(extend_tables), DKV_FAST(store_kv), DKV_FAST(attn_chunk),
                           DKV_FAST(attn_decode_window), {"load", load, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dkv_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dkv_call(void) {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&g_module) : nullptr;
}
