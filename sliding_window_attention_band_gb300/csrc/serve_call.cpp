// serve_call.cpp -- the serving calls of the binding without Python between the
// tensors and the library: a step of a small batch is three calls of a few
// microseconds on the GPU, and asking each tensor of a call its type, shape,
// place and address from Python takes longer than that (4.3 us a call; here
// 0.5).
//
// A function takes the address of the call's C descriptor, the tensors and
// what else the entry point takes.  It returns the library's status, or -1 when
// anything is not exactly as expected (a tensor of another type, shape, device
// or layout, a subclass, another current device): nothing has happened then,
// and the Python side looks again, tensor by tensor, and names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/TensorBase.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "swab.h"

namespace {

decltype(&rotary) fn_rotary;
decltype(&rotary_bwd) fn_rotary_bwd;
decltype(&cache_slots) fn_cache_slots;
decltype(&rotary_append) fn_rotary_append;
decltype(&band_decode) fn_band_decode;

// thrown (and caught at the entry) when a call has to be looked at again
struct Again {};

at::ScalarType type_of(int32_t dtype) {
    return dtype == SWAB_F32 ? at::kFloat : dtype == SWAB_F16 ? at::kHalf : at::kBFloat16;
}

// The tensors of one call: all plain, strided, on one CUDA device.
struct Call {
    int device = -1;

    const at::TensorBase &tensor(PyObject *o) {
        if (!THPVariable_CheckExact(o)) throw Again();
        const at::TensorBase &t = THPVariable_Unpack(o);
        if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) throw Again();
        if (device < 0) device = t.get_device();
        else if (t.get_device() != device) throw Again();
        return t;
    }
    template <typename P> P *contiguous(PyObject *o, at::ScalarType type, int64_t n, bool at_least = false) {
        const at::TensorBase &t = tensor(o);
        if (t.scalar_type() != type || !t.is_contiguous() || (at_least ? t.numel() < n : t.numel() != n)) throw Again();
        return static_cast<P *>(t.data_ptr());
    }
    int32_t *ints(PyObject *o, int64_t n, bool at_least = false) { return contiguous<int32_t>(o, at::kInt, n, at_least); }
    // a cache tensor [n_blocks, hk, page, hd]
    void *cache(PyObject *o, const swab_cache_desc &c, int hk, int hd, int32_t dtype) {
        const at::TensorBase &t = tensor(o);
        const auto s = t.sizes();
        if (t.scalar_type() != type_of(dtype) || s.size() != 4 || s[0] != c.n_blocks || s[1] != hk || s[2] != c.page || s[3] != hd ||
            !t.is_contiguous())
            throw Again();
        return t.data_ptr();
    }
    // heads of tokens [b, n, heads, hd] or [b * n, heads, hd], and their strides
    void *rows(PyObject *o, const swab_rotary_desc &d, int64_t heads, int64_t *stride) {
        const at::TensorBase &t = tensor(o);
        const auto s = t.sizes();
        const auto st = t.strides();
        const int64_t size[3] = {d.b, d.n, heads};
        if (t.scalar_type() != type_of(d.dtype)) throw Again();
        if (s.size() == 4 && s[0] == d.b && s[1] == d.n && s[2] == heads && s[3] == d.head_dim) {
            for (int k = 0; k < 3; ++k) stride[k] = st[k];
        } else if (s.size() == 3 && s[0] == (int64_t)d.b * d.n && s[1] == heads && s[2] == d.head_dim) {
            stride[0] = d.n * st[0];
            stride[1] = st[0];
            stride[2] = st[1];
        } else {
            throw Again();
        }
        bool any = false, many = false;
        for (int k = 0; k < 3; ++k) {
            if (size[k] == 1) stride[k] = 0;       // a single element's stride says nothing
            any |= stride[k] != 0;
            many |= size[k] > 1;
        }
        if (st[s.size() - 1] != 1 || (many && !any)) throw Again();
        return t.data_ptr();
    }
    // a tensor [tokens, h, hd] whose rows are row_stride (0: h * hd) apart
    void *heads(PyObject *o, const swab_decode_desc &d, int64_t row_stride) {
        const at::TensorBase &t = tensor(o);
        const auto s = t.sizes();
        if (t.scalar_type() != type_of(d.dtype) || s.size() != 3 || s[0] != d.tokens || s[1] != d.h || s[2] != d.head_dim)
            throw Again();
        if (row_stride != 0 || !t.is_contiguous()) {
            const auto st = t.strides();
            if (row_stride == 0) row_stride = (int64_t)d.h * d.head_dim;
            if ((st[0] != row_stride && s[0] > 1) || (st[1] != d.head_dim && s[1] > 1) || (st[2] != 1 && s[2] > 1)) throw Again();
        }
        return t.data_ptr();
    }
    uint64_t *turns(PyObject *o, const swab_rotary_desc &d) {
        return d.rot_dim == 0 ? nullptr : contiguous<uint64_t>(o, at::kLong, d.rot_dim / 2);
    }
    void *stream() {
        if (c10::cuda::current_device() != device) throw Again();
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    }
};

template <typename D> const D &desc(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p) throw Again();
    return *static_cast<const D *>(p);
}
int32_t number(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v != (int32_t)v) throw Again();
    return (int32_t)v;
}

template <typename F> swab_status without_gil(F &&f) {
    swab_status s;
    Py_BEGIN_ALLOW_THREADS
    s = f();
    Py_END_ALLOW_THREADS
    return s;
}

template <typename F> PyObject *entry(Py_ssize_t n, Py_ssize_t want, F &&f) {
    long rc = -1;
    if (n == want) {
        try {
            rc = (long)f();
        } catch (...) {        // Again, or an error of the tensor library: its own words come from the second look
            rc = -1;
        }
    }
    PyErr_Clear();
    return PyLong_FromLong(rc);
}

// (desc, turns, pos, Q, K, Qo, Ko); K, Ko are not looked at without key heads
template <bool kBackward> PyObject *py_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 7, [&] {
        swab_rotary_desc d = desc<swab_rotary_desc>(a[0]);
        Call c;
        void *q = c.rows(a[3], d, d.h, d.q_stride), *qo = c.rows(a[5], d, d.h, d.qo_stride), *k = nullptr, *ko = nullptr;
        if (d.hk > 0) {
            k = c.rows(a[4], d, d.hk, d.k_stride);
            ko = c.rows(a[6], d, d.hk, d.ko_stride);
        }
        const uint64_t *turns = c.turns(a[1], d);
        const int32_t *pos = a[2] == Py_None ? nullptr : c.ints(a[2], (int64_t)d.b * d.n);
        void *st = c.stream();
        return without_gil([&] { return (kBackward ? fn_rotary_bwd : fn_rotary)(&d, turns, pos, q, k, qo, ko, st); });
    });
}

// (cache, pos0, lens, n_new, table, free_list, used, lens_out, used_out, q_start, slots, pos)
PyObject *py_cache_slots(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 12, [&] {
        const swab_cache_desc &d = desc<swab_cache_desc>(a[0]);
        const int32_t pos0 = number(a[1]);
        Call c;
        const int64_t b = d.batch;
        const int32_t *lens = c.ints(a[2], b), *n_new = c.ints(a[3], b);
        int32_t *table = c.ints(a[4], b * d.cols);
        const int64_t n_free = c.tensor(a[5]).numel(), tokens = c.tensor(a[10]).numel();
        if (n_free > 0x7fffffff || tokens > 0x7fffffff) throw Again();
        const int32_t *free_list = c.ints(a[5], n_free), *used = c.ints(a[6], 1, true);
        int32_t *lens_out = c.ints(a[7], b), *used_out = c.ints(a[8], 2), *q_start = c.ints(a[9], b + 1);
        int32_t *slots = c.ints(a[10], tokens), *pos = c.ints(a[11], tokens);
        void *st = c.stream();
        return without_gil([&] {
            return fn_cache_slots(&d, (int32_t)tokens, pos0, lens, n_new, table, free_list, (int32_t)n_free, used, lens_out, used_out,
                                  q_start, slots, pos, st);
        });
    });
}

// (desc, cache, turns, Q, K, V, pos, slots, Qo, Kc, Vc)
PyObject *py_rotary_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 11, [&] {
        swab_rotary_desc d = desc<swab_rotary_desc>(a[0]);
        const swab_cache_desc &cache = desc<swab_cache_desc>(a[1]);
        if ((a[3] == Py_None) != (a[8] == Py_None)) throw Again();
        Call c;
        void *k = c.rows(a[4], d, d.hk, d.k_stride), *v = c.rows(a[5], d, d.hk, d.v_stride), *q = nullptr, *qo = nullptr;
        if (a[3] != Py_None) {
            q = c.rows(a[3], d, d.h, d.q_stride);
            qo = c.rows(a[8], d, d.h, d.qo_stride);
        }
        const uint64_t *turns = c.turns(a[2], d);
        const int64_t tokens = (int64_t)d.b * d.n;
        const int32_t *pos = a[6] == Py_None ? nullptr : c.ints(a[6], tokens), *slots = c.ints(a[7], tokens);
        void *kc = c.cache(a[9], cache, d.hk, d.head_dim, d.dtype), *vc = c.cache(a[10], cache, d.hk, d.head_dim, d.dtype);
        void *st = c.stream();
        return without_gil([&] { return fn_rotary_append(&d, &cache, turns, pos, slots, q, k, v, qo, kc, vc, st); });
    });
}

// (desc, need, scale, Q, Kc, Vc, table, lens, q_start, prefix_table, O, lse, workspace); need: bytes of workspace
PyObject *py_band_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 13, [&] {
        const swab_decode_desc &d = desc<swab_decode_desc>(a[0]);
        const long long need = PyLong_AsLongLong(a[1]);
        if (!PyFloat_Check(a[2]) && !PyLong_Check(a[2])) throw Again();
        const double scale = PyFloat_AsDouble(a[2]);
        if (PyErr_Occurred()) throw Again();
        const swab_cache_desc &cd = d.cache;
        Call c;
        void *q = c.heads(a[3], d, d.q_row_stride), *o = c.heads(a[10], d, d.out_row_stride);
        void *kc = c.cache(a[4], cd, d.hk, d.head_dim, d.dtype), *vc = c.cache(a[5], cd, d.hk, d.head_dim, d.dtype);
        const int32_t *table = c.ints(a[6], (int64_t)cd.batch * cd.cols), *lens = c.ints(a[7], cd.batch),
                      *q_start = c.ints(a[8], (int64_t)cd.batch + 1), *ptable = nullptr;
        if (d.prefix_len > 0) ptable = c.ints(a[9], ((int64_t)d.prefix_len + cd.page - 1) / cd.page);
        float *lse = nullptr;
        if (a[11] != Py_None) {
            lse = c.contiguous<float>(a[11], at::kFloat, (int64_t)d.tokens * d.h);
            const auto s = c.tensor(a[11]).sizes();
            if (s.size() != 2 || s[0] != d.tokens) throw Again();
        }
        void *ws = nullptr;
        if (need > 0) {
            const at::TensorBase &t = c.tensor(a[12]);
            if ((long long)t.nbytes() < need || !t.is_contiguous()) throw Again();
            ws = t.data_ptr();
        }
        void *st = c.stream();
        return without_gil([&] { return fn_band_decode(&d, (float)scale, q, kc, vc, table, lens, q_start, ptable, o, lse, ws, st); });
    });
}

// bind(rotary, rotary_bwd, cache_slots, rotary_append, band_decode): the library's entry points by address
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind: five addresses expected");
        return nullptr;
    }
    void *p[5];
    for (int k = 0; k < 5; ++k)
        if (!(p[k] = PyLong_AsVoidPtr(a[k]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: an address is null");
            return nullptr;
        }
    fn_rotary = reinterpret_cast<decltype(fn_rotary)>(p[0]);
    fn_rotary_bwd = reinterpret_cast<decltype(fn_rotary_bwd)>(p[1]);
    fn_cache_slots = reinterpret_cast<decltype(fn_cache_slots)>(p[2]);
    fn_rotary_append = reinterpret_cast<decltype(fn_rotary_append)>(p[3]);
    fn_band_decode = reinterpret_cast<decltype(fn_band_decode)>(p[4]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(py_bind)},
                         {"rotary", FAST(py_rotary<false>)},
                         {"rotary_bwd", FAST(py_rotary<true>)},
                         {"cache_slots", FAST(py_cache_slots)},
                         {"rotary_append", FAST(py_rotary_append)},
                         {"band_decode", FAST(py_band_decode)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_call(void) { return PyModule_Create(&module); }
