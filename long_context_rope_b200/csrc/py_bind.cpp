// py_bind.cpp -- the Python side's fast path into libhga.so: a tensor's checks
// in one call, and the calls themselves without ctypes' conversions. A decode
// loop's host time is mostly these: a call with five tensors spent 4.6 us on
// them in Python and ctypes, 0.6 us here.
//
// ptr(t, name, dtype=None, shape=None, device=True, nullable=False): the tensor's
// address if it is as asked; whatever else goes on to the Python function given
// to set_refuse, which finds out what is wrong and raises.
// shape_key(cfg, windows): the bytes of the hga_config at address cfg, but in the place of
// q_begin the number of chunks that the span touches, and with windows seq_len 0.
// hga_*(...): as declared in hga.h; pointers are integers or None.
#include <Python.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <utility>

#include "hga.h"

namespace {

PyObject* g_refuse = nullptr;

bool as_asked(PyObject* t, PyObject* dtype, PyObject* shape, bool device, void** out) {
    if (!THPVariable_Check(t)) return false;
    const at::Tensor& x = THPVariable_Unpack(t);
    if (dtype != Py_None &&
        !(THPDtype_Check(dtype) &&
          reinterpret_cast<THPDtype*>(dtype)->scalar_type == x.scalar_type()))
        return false;
    if (shape != Py_None) {
        if (!PyTuple_Check(shape)) return false;
        const auto sizes = x.sizes();
        if (PyTuple_GET_SIZE(shape) != (Py_ssize_t)sizes.size()) return false;
        for (size_t i = 0; i < sizes.size(); ++i) {
            const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, (Py_ssize_t)i));
            if (n == -1 && PyErr_Occurred()) {
                PyErr_Clear();
                return false;
            }
            if (n != sizes[i]) return false;
        }
    }
    if (!x.is_contiguous()) return false;
    if (device && !(x.is_cuda() &&
                    x.get_device() ==
                        c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index()))
        return false;
    *out = x.data_ptr();
    return true;
}

constexpr const char* kPtrArgs[] = {"t", "name", "dtype", "shape", "device", "nullable"};

PyObject* ptr(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    PyObject* a[6] = {nullptr, nullptr, Py_None, Py_None, Py_True, Py_False};
    bool known = n <= 6;
    for (Py_ssize_t i = 0; known && i < n; ++i) a[i] = args[i];
    const Py_ssize_t n_kw = kw ? PyTuple_GET_SIZE(kw) : 0;
    for (Py_ssize_t k = 0; known && k < n_kw; ++k) {
        known = false;
        for (int i = 0; i < 6; ++i)
            if (PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(kw, k), kPtrArgs[i]) == 0) {
                a[i] = args[n + k];
                known = true;
            }
    }
    if (known && a[0] && a[1]) {
        if (a[0] == Py_None && a[5] == Py_True) Py_RETURN_NONE;
        void* p;
        try {
            if (as_asked(a[0], a[2], a[3], a[4] == Py_True, &p)) return PyLong_FromVoidPtr(p);
        } catch (...) {  // a tensor without storage, say: Python's own calls say so
        }
    }
    if (!g_refuse) {
        PyErr_SetString(PyExc_RuntimeError, "set_refuse was not called");
        return nullptr;
    }
    return PyObject_Vectorcall(g_refuse, args, (size_t)n, kw);
}

PyObject* set_refuse(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(g_refuse, f);
    Py_RETURN_NONE;
}

PyObject* shape_key(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "2 arguments, not %zd", n);
    const auto* at = static_cast<const hga_config*>(PyLong_AsVoidPtr(args[0]));
    if (!at) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no configuration");
        return nullptr;
    }
    PyObject* out = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(at), sizeof(*at));
    if (!out) return nullptr;
    auto* c = reinterpret_cast<hga_config*>(PyBytes_AS_STRING(out));
    const int64_t first = c->q_begin, last = first + c->q_len - 1, size = c->chunk_size;
    auto chunk = [size](int64_t t) { return t / size - (t % size < 0 ? 1 : 0); };
    c->q_begin = c->q_len < 1 || size < 1 ? 0 : (int32_t)(chunk(last) - chunk(first) + 1);
    if (args[1] == Py_True) c->seq_len = 0;
    return out;
}

template <typename T>
bool get(PyObject* o, T*& v) {
    v = nullptr;
    if (o == Py_None) return true;
    v = reinterpret_cast<T*>(PyLong_AsVoidPtr(o));
    return v || !PyErr_Occurred();
}
bool get(PyObject* o, int64_t& v) {
    v = PyLong_AsLongLong(o);
    return v != -1 || !PyErr_Occurred();
}
bool get(PyObject* o, int32_t& v) {
    int64_t w;
    if (!get(o, w)) return false;
    v = (int32_t)w;
    if (v == w) return true;
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return false;
}

template <auto F>
struct Entry;
template <typename... A, hga_status (*F)(A...)>
struct Entry<F> {
    template <size_t... I>
    static bool convert(PyObject* const* a, std::tuple<A...>& v, std::index_sequence<I...>) {
        return (get(a[I], std::get<I>(v)) && ...);
    }
    static PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
        if (n != (Py_ssize_t)sizeof...(A))
            return PyErr_Format(PyExc_TypeError, "%zu arguments, not %zd", sizeof...(A), n);
        std::tuple<A...> v;
        if (!convert(a, v, std::index_sequence_for<A...>())) return nullptr;
        hga_status s;
        Py_BEGIN_ALLOW_THREADS;
        s = std::apply(F, v);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(s);
    }
};

#define HGA_ENTRY(f) {#f, (PyCFunction)(void (*)(void))Entry<f>::call, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    {"ptr", (PyCFunction)(void (*)(void))ptr, METH_FASTCALL | METH_KEYWORDS,
     "Address of a tensor that has the type, shape, place and layout asked for."},
    {"set_refuse", set_refuse, METH_O, "What ptr goes on to for any other argument."},
    {"shape_key", (PyCFunction)(void (*)(void))shape_key, METH_FASTCALL,
     "A configuration's bytes, the same wherever its span of as many chunks lies."},
    HGA_ENTRY(hga_apply_rope),
    HGA_ENTRY(hga_apply_rope_axes),
    HGA_ENTRY(hga_build_summaries),
    HGA_ENTRY(hga_build_summaries_axes),
    HGA_ENTRY(hga_store_kv),
    HGA_ENTRY(hga_load_kv),
    HGA_ENTRY(hga_route_chunks),
    HGA_ENTRY(hga_route_groups),
    HGA_ENTRY(hga_route),
    HGA_ENTRY(hga_decode_step),
    HGA_ENTRY(hga_decode_step_tiered),
    HGA_ENTRY(hga_gather_kv),
    HGA_ENTRY(hga_gather_kv_warm),
    HGA_ENTRY(hga_gather_kv_warm_noalloc),
    HGA_ENTRY(hga_attend),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_hga_bind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the versions of torch and Python whose headers this was compiled with.
PyMODINIT_FUNC PyInit__hga_bind(void) {
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", HGA_BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
