// binding.cpp -- the quick way into the serving entry points from Python.
//
// A decoding step calls fa_rope, fa_kv_append and fa_fwd_paged with a dozen tensors each, on
// work of a few microseconds; checked in Python and marshalled by ctypes a call took 9 to 12
// us of host time.  These functions make the same checks on the tensors' C++ objects and call
// the C entry point by its address.  They decide nothing: a call that is not plain (an
// argument of another kind, shape, type or device, the tensors' device not current) returns
// None, and the caller goes on to the checks in Python, which name what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

// (called by address: the library is loaded by the caller)
using RopeFn = decltype(&fa_rope);
using AppendFn = decltype(&fa_kv_append);
using PagedFn = decltype(&fa_fwd_paged);

// A [n0, n1, n2, d] tensor with d contiguous.
struct Rows {
    void *p = nullptr;
    int64_t n[4] = {0, 0, 0, 0};
    long long st[3];
    const long long *strides = nullptr;  // nullptr: contiguous
};

struct Call {
    at::ScalarType type = at::ScalarType::Undefined;
    int device = -1;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o) {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // The call's first tensor sets its type and device.
    void rows(PyObject *o, Rows &r, bool first = false) {
        const at::Tensor *t = tensor(o);
        if (!t) return;
        if (first) {
            type = t->scalar_type();
            if (!t->is_cuda() || (type != at::kBFloat16 && type != at::kHalf)) {
                ok = false;
                return;
            }
            device = t->get_device();
        }
        if (!t->is_cuda() || t->dim() != 4 || t->scalar_type() != type || t->get_device() != device) {
            ok = false;
            return;
        }
        for (int i = 0; i < 4; ++i) {
            r.n[i] = t->size(i);
            if (r.n[i] > INT_MAX) ok = false;
        }
        if (!t->is_contiguous()) {
            if (t->stride(3) != 1) ok = false;
            for (int i = 0; i < 3; ++i) r.st[i] = t->stride(i);
            r.strides = r.st;
        }
        r.p = t->data_ptr();
    }
    // A contiguous tensor of another type; nullptr for None.
    void *plain(PyObject *o, at::ScalarType ty, std::initializer_list<int64_t> shape) {
        const at::Tensor *t = tensor(o);
        if (!t) return nullptr;
        if (!t->is_cuda() || t->scalar_type() != ty || t->get_device() != device || !t->is_contiguous() ||
            t->sizes() != at::IntArrayRef(shape))
            ok = false;
        return t->data_ptr();
    }
    void same(const Rows &a, const Rows &b) {
        for (int i = 0; i < 4; ++i) ok = ok && a.n[i] == b.n[i];
    }
    int dtype() const { return type == at::kBFloat16 ? 0 : 1; }
    // The stream handle given (an integer), or the device's current one for None.
    void *stream(PyObject *o) {
        if (!ok || c10::cuda::current_device() != device) {
            ok = false;
            return nullptr;
        }
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
        if (!PyLong_Check(o)) {
            ok = false;
            return nullptr;
        }
        return PyLong_AsVoidPtr(o);
    }
};

struct Plan {
    const unsigned long long *turns = nullptr;
    int rot = 0, inter = 0;
    float mag = 1.f;
    // a = (turns, rot_dim, interleaved, magnitude)
    void read(Call &c, PyObject *const *a) {
        rot = (int)PyLong_AsLong(a[1]);
        inter = PyObject_IsTrue(a[2]) ? 1 : 0;
        mag = (float)PyFloat_AsDouble(a[3]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            c.ok = false;
        }
        turns = static_cast<unsigned long long *>(c.plain(a[0], at::kLong, {rot / 2}));
    }
};

template <typename F>
F address(PyObject *o) {
    return reinterpret_cast<F>(PyLong_AsVoidPtr(o));
}

PyObject *answer(const Call &c, int rc) {
    if (!c.ok) Py_RETURN_NONE;
    return PyLong_FromLong(rc);
}

// rope(address, x, x_out, y, y_out, positions, turns, rot_dim, interleaved, magnitude, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11) Py_RETURN_NONE;
    Call c;
    Rows x, xo, y, yo;
    c.rows(a[1], x, true);
    c.rows(a[2], xo);
    if (c.ok) c.same(x, xo);
    const bool two = a[3] != Py_None;
    if (two != (a[4] != Py_None)) Py_RETURN_NONE;
    if (two && c.ok) {
        c.rows(a[3], y);
        c.rows(a[4], yo);
        c.same(y, yo);
        c.ok = c.ok && y.n[0] == x.n[0] && y.n[2] == x.n[2] && y.n[3] == x.n[3];
    }
    const int *pos = nullptr;
    int per_batch = 0;
    if (a[5] != Py_None && c.ok) {
        const at::Tensor *t = c.tensor(a[5]);
        per_batch = t && t->dim() == 2;
        pos = static_cast<int *>(per_batch ? c.plain(a[5], at::kInt, {x.n[0], x.n[2]})
                                           : c.plain(a[5], at::kInt, {x.n[2]}));
    }
    Plan plan;
    if (c.ok) plan.read(c, a + 6);
    void *st = c.stream(a[10]);
    int rc = 0;
    if (c.ok)
        rc = address<RopeFn>(a[0])(x.p, xo.p, y.p, yo.p, (int)x.n[0], (int)x.n[1], (int)y.n[1],
                                   (int)x.n[2], (int)x.n[3], x.strides, xo.strides, y.strides,
                                   yo.strides, pos, per_batch, plan.turns, plan.rot, plan.inter,
                                   plan.mag, c.dtype(), st);
    return answer(c, rc);
}

// A cache with its table and lengths.
struct Cache {
    Rows k, v;
    int *table = nullptr, *held = nullptr, *fresh = nullptr;
    int blocks = 0;
    // a = (k_cache, v_cache, block_table, cache_len, new_len)
    void read(Call &c, PyObject *const *a, int64_t B, int64_t d) {
        c.rows(a[0], k);
        c.rows(a[1], v);
        if (!c.ok) return;
        c.same(k, v);
        c.ok = c.ok && k.n[3] == d;
        const at::Tensor *t = c.tensor(a[2]);
        if (!t || t->dim() != 2) {
            c.ok = false;
            return;
        }
        if (t->size(1) > INT_MAX) c.ok = false;
        blocks = (int)t->size(1);
        table = static_cast<int *>(c.plain(a[2], at::kInt, {B, t->size(1)}));
        held = static_cast<int *>(c.plain(a[3], at::kInt, {B}));
        if (a[4] != Py_None) fresh = static_cast<int *>(c.plain(a[4], at::kInt, {B}));
    }
};

// append(address, k, v, k_cache, v_cache, block_table, cache_len, new_len, q, q_out, positions,
//        turns, rot_dim, interleaved, magnitude, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 16) Py_RETURN_NONE;
    Call c;
    Rows k, v, q, qo;
    c.rows(a[1], k, true);
    c.rows(a[2], v);
    if (c.ok) c.same(k, v);
    Cache cache;
    if (c.ok) cache.read(c, a + 3, k.n[0], k.n[3]);
    c.ok = c.ok && cache.k.n[1] == k.n[1];
    const bool two = a[8] != Py_None;
    if (two != (a[9] != Py_None)) Py_RETURN_NONE;
    if (two && c.ok) {
        c.rows(a[8], q);
        c.rows(a[9], qo);
        c.same(q, qo);
        c.ok = c.ok && q.n[0] == k.n[0] && q.n[2] == k.n[2] && q.n[3] == k.n[3];
    }
    const int *pos = nullptr;
    if (a[10] != Py_None && c.ok) pos = static_cast<int *>(c.plain(a[10], at::kInt, {k.n[0], k.n[2]}));
    Plan plan;
    if (a[11] != Py_None && c.ok) plan.read(c, a + 11);
    void *st = c.stream(a[15]);
    int rc = 0;
    if (c.ok)
        rc = address<AppendFn>(a[0])(
            k.p, v.p, cache.k.p, cache.v.p, q.p, qo.p, (int)k.n[0], (int)q.n[1], (int)k.n[1],
            (int)k.n[2], (int)k.n[3], k.strides, v.strides, q.strides, qo.strides, cache.k.strides,
            cache.v.strides, (int)cache.k.n[0], (int)cache.k.n[2], cache.table, cache.blocks,
            cache.held, cache.fresh, pos, plan.turns, plan.rot, plan.inter, plan.mag, c.dtype(), st);
    return answer(c, rc);
}

// paged(address, q, k_cache, v_cache, block_table, cache_len, new_len, o, lse, tree_mask,
//       workspace, scale, stream)
PyObject *paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13) Py_RETURN_NONE;
    Call c;
    Rows q, o;
    c.rows(a[1], q, true);
    c.rows(a[7], o);
    if (c.ok) c.same(q, o);
    Cache cache;
    if (c.ok) cache.read(c, a + 2, q.n[0], q.n[3]);
    float *lse = nullptr;
    unsigned char *tree = nullptr;
    int per_batch = 0;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (c.ok) {
        lse = static_cast<float *>(c.plain(a[8], at::kFloat, {q.n[0], q.n[1], q.n[2]}));
        if (a[9] != Py_None) {
            const at::Tensor *t = c.tensor(a[9]);
            per_batch = t && t->dim() == 3;
            tree = static_cast<unsigned char *>(per_batch ? c.plain(a[9], at::kByte, {q.n[0], q.n[2], q.n[2]})
                                                          : c.plain(a[9], at::kByte, {q.n[2], q.n[2]}));
        }
        const at::Tensor *t = c.tensor(a[10]);
        if (t && t->is_cuda() && t->scalar_type() == at::kByte && t->get_device() == c.device &&
            t->is_contiguous()) {
            ws = t->data_ptr();
            ws_bytes = (size_t)t->numel();
        } else {
            c.ok = false;
        }
    }
    const double scale = PyFloat_AsDouble(a[11]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c.ok = false;
    }
    void *st = c.stream(a[12]);
    int rc = 0;
    if (c.ok)
        rc = address<PagedFn>(a[0])(
            q.p, cache.k.p, cache.v.p, o.p, lse, (int)q.n[0], (int)q.n[1], (int)cache.k.n[1],
            (int)q.n[2], (int)q.n[3], q.strides, o.strides, cache.k.strides, cache.v.strides,
            (int)cache.k.n[0], (int)cache.k.n[2], cache.table, cache.blocks, cache.held, cache.fresh,
            tree, per_batch, (float)scale, c.dtype(), ws, ws_bytes, st);
    return answer(c, rc);
}

// No C++ exception leaves a call: it becomes None (the checks in Python say what is wrong).
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<rope>)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<append>)), METH_FASTCALL, nullptr},
    {"paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<paged>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch version whose headers this was compiled against.
PyMODINIT_FUNC PyInit__fa_binding() {
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FA_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
