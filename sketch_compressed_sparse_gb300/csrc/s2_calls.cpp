// Python's way into the 8-bit layer's calls of libs2. They are the functions
// that ctypes calls, with the same arguments; converting ten to fourteen of
// them is what ctypes takes 1.1 to 1.3 us for, and a call of a token's size is
// not much longer than that.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "s2.h"
#include "s2_header_id.h"

namespace {

decltype(&s2_pack8) pack8;
decltype(&s2_unpack8) unpack8;
decltype(&s2_matmul8) matmul8;
decltype(&s2_wgrad8) wgrad8;

// Positional arguments: integers, and None for a null pointer.
struct In {
    PyObject* const* v;
    bool bad = false;
    uint64_t u(int i) {
        if (v[i] == Py_None) return 0;
        const uint64_t x = PyLong_AsUnsignedLongLong(v[i]);
        bad |= x == ~0ull && PyErr_Occurred();
        return x;
    }
    int n(int i) {
        const long x = PyLong_AsLong(v[i]);
        bad |= x == -1 && PyErr_Occurred();
        return (int)x;
    }
    template <typename T>
    T* p(int i) {
        return reinterpret_cast<T*>(u(i));
    }
    s2_dtype dtype(int i) { return (s2_dtype)n(i); }
    s2_scale_layout layout(int i) { return (s2_scale_layout)n(i); }
};

// The status of f(args...), called without the interpreter's lock.
template <typename F, typename... A>
PyObject* status_of(bool bad, F f, A... args) {
    if (bad) return nullptr;
    s2_status st;
    Py_BEGIN_ALLOW_THREADS st = f(args...);
    Py_END_ALLOW_THREADS return PyLong_FromLong(st);
}
bool wants(Py_ssize_t given, Py_ssize_t wanted) {
    if (given == wanted) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", given, wanted);
    return false;
}

PyObject* py_pack8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (!wants(n, 13)) return nullptr;
    In a{v};
    const void* x = a.p<void>(0);
    const s2_dtype dt = a.dtype(1);
    const uint64_t rows = a.u(2), cols = a.u(3), ldx = a.u(4);
    const s2_scale_layout lay = a.layout(5);
    uint8_t* codes = a.p<uint8_t>(6);
    const uint64_t ldc = a.u(7);
    uint8_t *scales = a.p<uint8_t>(8), *codes_t = a.p<uint8_t>(9);
    const uint64_t ldct = a.u(10);
    uint8_t* scales_t = a.p<uint8_t>(11);
    const auto stream = (s2_stream_t)a.p<void>(12);
    return status_of(a.bad, pack8, x, dt, rows, cols, ldx, lay, codes, ldc, scales, codes_t, ldct, scales_t, stream);
}

PyObject* py_unpack8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (!wants(n, 10)) return nullptr;
    In a{v};
    const uint8_t* codes = a.p<uint8_t>(0);
    const uint64_t ldc = a.u(1);
    const uint8_t* scales = a.p<uint8_t>(2);
    const s2_scale_layout lay = a.layout(3);
    const uint64_t rows = a.u(4), cols = a.u(5);
    void* out = a.p<void>(6);
    const s2_dtype dt = a.dtype(7);
    const uint64_t ldo = a.u(8);
    const auto stream = (s2_stream_t)a.p<void>(9);
    return status_of(a.bad, unpack8, codes, ldc, scales, lay, rows, cols, out, dt, ldo, stream);
}

PyObject* py_matmul8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (!wants(n, 14)) return nullptr;
    In a{v};
    const uint8_t* x = a.p<uint8_t>(0);
    const uint64_t ldx = a.u(1);
    const uint8_t *xs = a.p<uint8_t>(2), *w = a.p<uint8_t>(3);
    const uint64_t ldw = a.u(4);
    const uint8_t* ws = a.p<uint8_t>(5);
    const s2_scale_layout lay = a.layout(6);
    const uint64_t M = a.u(7), N = a.u(8), K = a.u(9);
    void* y = a.p<void>(10);
    const s2_dtype dt = a.dtype(11);
    const uint64_t ldy = a.u(12);
    const auto stream = (s2_stream_t)a.p<void>(13);
    return status_of(a.bad, matmul8, x, ldx, xs, w, ldw, ws, lay, M, N, K, y, dt, ldy, stream);
}

PyObject* py_wgrad8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (!wants(n, 13)) return nullptr;
    In a{v};
    const void* dy = a.p<void>(0);
    const uint64_t lddy = a.u(1);
    const uint8_t* x = a.p<uint8_t>(2);
    const uint64_t ldx = a.u(3);
    const uint8_t* xs = a.p<uint8_t>(4);
    const uint64_t T = a.u(5), N = a.u(6), K = a.u(7);
    void* dw = a.p<void>(8);
    const s2_dtype dt = a.dtype(9);
    const uint64_t lddw = a.u(10);
    const int accumulate = a.n(11);
    const auto stream = (s2_stream_t)a.p<void>(12);
    return status_of(a.bad, wgrad8, dy, lddy, x, ldx, xs, T, N, K, dw, dt, lddw, accumulate, stream);
}

// bind(s2_pack8, s2_unpack8, s2_matmul8, s2_wgrad8): their addresses in the loaded library.
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (!wants(n, 4)) return nullptr;
    In a{v};
    const uint64_t at[4] = {a.u(0), a.u(1), a.u(2), a.u(3)};
    if (a.bad) return nullptr;
    pack8 = reinterpret_cast<decltype(pack8)>(at[0]);
    unpack8 = reinterpret_cast<decltype(unpack8)>(at[1]);
    matmul8 = reinterpret_cast<decltype(matmul8)>(at[2]);
    wgrad8 = reinterpret_cast<decltype(wgrad8)>(at[3]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<py_bind>("bind"),       method<py_pack8>("s2_pack8"),   method<py_unpack8>("s2_unpack8"),
                         method<py_matmul8>("s2_matmul8"), method<py_wgrad8>("s2_wgrad8"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_s2calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__s2calls() {
    PyObject* m = PyModule_Create(&module);
    // the library's version ends with the same word where both are of one header
    if (m && PyModule_AddStringConstant(m, "header", S2_HEADER_WORD) < 0) Py_CLEAR(m);
    return m;
}
