// Host side of the serving calls as a CPython module over torch's tensors.
// These calls are shorter on the GPU than the interpreter needs to look at
// their arguments one attribute at a time (mx_gemv 8.1 us of host time,
// mx_cache_attention 11.8, of which the launch is 3.3), so the usual call is
// checked and packed here.  A function returns
//   - its result, or
//   - an int: the status that the C ABI refused the call with, or
//   - None for anything but the usual call (an argument that is no GPU tensor
//     of the right type and shape, bf16 given as bits, strides that are
//     refused, a workspace of the caller's).  The Python side then looks at
//     the arguments itself: it words the errors, and takes the rest.
// Nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kroquant.h"

namespace {

decltype(&mx_gemv) gemv_fn;
decltype(&mx_cache_write) write_fn;
decltype(&mx_cache_read) read_fn;
decltype(&mx_cache_attention) attention_fn;
decltype(&mx_cache_attention_workspace) workspace_fn;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous GPU tensor of the type, or null.
const at::Tensor *plain(PyObject *o, at::ScalarType type)
{
    const at::Tensor *t = tensor(o);
    return t && t->is_cuda() && t->scalar_type() == type && t->layout() == at::kStrided && t->is_contiguous() ? t
                                                                                                             : nullptr;
}

bool whole(PyObject *o, int64_t &v)
{
    if (!PyLong_CheckExact(o))
        return false;
    int over = 0;
    v = PyLong_AsLongLongAndOverflow(o, &over);
    return over == 0;
}

void *handle(PyObject *o) { return (void *)PyLong_AsUnsignedLongLong(o); }

at::Tensor fresh(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType type)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

PyObject *none() { Py_RETURN_NONE; }

// The cache's tensors and sizes; false: not the usual call.
bool read_cache(PyObject *o, mx_cache &c, const at::Tensor *&kq)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
        return false;
    const at::Tensor *t[4];
    for (int i = 0; i < 4; ++i)
        if (!(t[i] = plain(PyTuple_GET_ITEM(o, i), at::kByte)) || t[i]->dim() != 4)
            return false;
    const auto q = t[0]->sizes(), s = t[1]->sizes();
    if (t[2]->sizes() != q || t[3]->sizes() != s || s[0] != q[0] || s[1] != q[1] || s[2] != q[3] / 16 || s[3] != q[2])
        return false;
    c = {(uint8_t *)t[0]->data_ptr(), (uint8_t *)t[1]->data_ptr(), (uint8_t *)t[2]->data_ptr(),
         (uint8_t *)t[3]->data_ptr(), q[0], q[2], q[1], 2 * q[3]};
    kq = t[0];
    return true;
}

bool read_batch(PyObject *table, PyObject *start, PyObject *lengths, int64_t rows, mx_batch &b)
{
    const at::Tensor *t = plain(table, at::kInt), *s = plain(start, at::kInt), *l = plain(lengths, at::kInt);
    if (!t || !s || !l || t->dim() != 2 || t->size(0) != l->numel() || s->numel() != l->numel() + 1)
        return false;
    b = {(const int32_t *)t->data_ptr(), (const int32_t *)s->data_ptr(), (const int32_t *)l->data_ptr(), l->numel(),
         t->size(1), rows};
    return true;
}

// A bf16 [rows, heads, dim] view whose rows are dense inside.
const at::Tensor *heads_view(PyObject *o, int64_t dim, int64_t &stride)
{
    const at::Tensor *t = tensor(o);
    if (!t || !t->is_cuda() || t->scalar_type() != at::kBFloat16 || t->layout() != at::kStrided || t->dim() != 3 ||
        t->size(2) != dim || t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != dim))
        return nullptr;
    stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * dim;
    return t;
}

// torch's exceptions (no memory left, say) as Python's.
PyObject *guarded(PyObject *(*f)(PyObject *const *), PyObject *const *a)
{
    HANDLE_TH_ERRORS
    return f(a);
    END_HANDLE_TH_ERRORS
}

// Other Python threads run while a launch is queued.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class F, class... A>
int call(F f, A... a)
{
    const Unlocked unlocked;
    return f(a...);
}

// x, qw, sw, out or None, bf16 out (0 / 1; with out given: as out is), stream
PyObject *gemv(PyObject *const *a)
{
    const at::Tensor *x = plain(a[0], at::kBFloat16), *qw = plain(a[1], at::kByte), *sw = plain(a[2], at::kByte);
    if (!x || !qw || !sw || x->dim() != 2 || qw->dim() != 2 || sw->dim() != 2)
        return none();
    const int64_t M = x->size(0), K = x->size(1), N = qw->size(0);
    if (qw->size(1) != K / 2 || sw->size(0) != N || sw->size(1) != K / 32)
        return none();
    const bool bf16 = a[4] == Py_True;
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
    at::Tensor made;
    const at::Tensor *out = &made;
    if (a[3] == Py_None)
        made = fresh(*x, {M, N}, type);
    else if (!(out = plain(a[3], type)) || out->dim() != 2 || out->size(0) != M || out->size(1) != N)
        return none();
    const int st = call(gemv_fn, (const uint16_t *)x->data_ptr(), M, (const uint8_t *)qw->data_ptr(),
                           (const uint8_t *)sw->data_ptr(), N, K, out->data_ptr(), bf16, handle(a[5]));
    if (st)
        return PyLong_FromLong(st);
    return a[3] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[3]);
}

// k, v, cache, page_table, row_start, lengths, factors or None, stream; True when done
PyObject *write(PyObject *const *a)
{
    mx_cache c;
    mx_batch b;
    const at::Tensor *kq, *f = nullptr;
    if (!read_cache(a[2], c, kq))
        return none();
    int64_t ks, vs;
    const at::Tensor *k = heads_view(a[0], c.dim, ks), *v = heads_view(a[1], c.dim, vs);
    if (!k || !v || k->size(1) != c.heads || v->size(1) != c.heads || k->size(0) != v->size(0) ||
        !read_batch(a[3], a[4], a[5], k->size(0), b))
        return none();
    if (a[6] != Py_None && (!(f = plain(a[6], at::kFloat)) || f->numel() % 20 != 0))
        return none();
    const int st = call(write_fn, (const uint16_t *)k->data_ptr(), ks, (const uint16_t *)v->data_ptr(), vs,
                            f ? (const float *)f->data_ptr() : nullptr, f ? f->numel() / 20 : 1, &c, &b, handle(a[7]));
    if (st)
        return PyLong_FromLong(st);
    Py_RETURN_TRUE;
}

// cache, page_table, row_start, lengths, rows, stream; (k, v)
PyObject *read(PyObject *const *a)
{
    mx_cache c;
    mx_batch b;
    const at::Tensor *kq;
    int64_t rows;
    if (!whole(a[4], rows) || rows < 0 || !read_cache(a[0], c, kq) || !read_batch(a[1], a[2], a[3], rows, b))
        return none();
    at::Tensor k = fresh(*kq, {rows, c.heads, c.dim}, at::kBFloat16), v = fresh(*kq, {rows, c.heads, c.dim}, at::kBFloat16);
    const int st = call(read_fn, &c, &b, (uint16_t *)k.data_ptr(), (uint16_t *)v.data_ptr(), handle(a[5]));
    if (st)
        return PyLong_FromLong(st);
    PyObject *pair = PyTuple_New(2);
    if (pair) {
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(k)));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(v)));
    }
    return pair;
}

// q, cache, page_table, row_start, lengths, scale or None, window, sinks, out or None, stream
PyObject *attention(PyObject *const *a)
{
    mx_cache c;
    mx_batch b;
    const at::Tensor *kq;
    int64_t qs, os, window, sinks;
    if (!read_cache(a[1], c, kq) || !whole(a[6], window) || !whole(a[7], sinks) ||
        (a[5] != Py_None && !PyFloat_CheckExact(a[5])))
        return none();
    const at::Tensor *q = heads_view(a[0], c.dim, qs);
    if (!q || !read_batch(a[2], a[3], a[4], q->size(0), b))
        return none();
    const int64_t heads = q->size(1);
    int64_t need = 0;
    int st = workspace_fn(heads, &c, &b, window, sinks, &need);
    if (st)
        return PyLong_FromLong(st);
    at::Tensor made, work;
    const at::Tensor *out = &made;
    if (a[8] == Py_None) {
        made = fresh(*q, q->sizes(), at::kBFloat16);
        os = heads * c.dim;
    } else if (!(out = heads_view(a[8], c.dim, os)) || out->sizes() != q->sizes()) {
        return none();
    }
    if (need)
        work = fresh(*q, {need}, at::kByte);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)c.dim) : PyFloat_AS_DOUBLE(a[5]);
    st = call(attention_fn, (const uint16_t *)q->data_ptr(), qs, heads, &c, &b, (float)scale, window, sinks,
                      (uint16_t *)out->data_ptr(), os, need ? work.data_ptr() : nullptr, need, handle(a[9]));
    if (st)
        return PyLong_FromLong(st);
    return a[8] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[8]);
}

template <PyObject *(*f)(PyObject *const *), int n>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (count != n) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    return guarded(f, a);
}

// The addresses of the C ABI's functions, from the library that is loaded.
PyObject *bind(PyObject *const *a)
{
    gemv_fn = (decltype(gemv_fn))handle(a[0]);
    write_fn = (decltype(write_fn))handle(a[1]);
    read_fn = (decltype(read_fn))handle(a[2]);
    attention_fn = (decltype(attention_fn))handle(a[3]);
    workspace_fn = (decltype(workspace_fn))handle(a[4]);
    return none();
}

#define KQ_ENTRY(name, count) {#name, (PyCFunction)(void (*)(void))entry<name, count>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KQ_ENTRY(bind, 5),  KQ_ENTRY(gemv, 6),       KQ_ENTRY(write, 8),
                         KQ_ENTRY(read, 6),  KQ_ENTRY(attention, 10), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods};

} // namespace

PyMODINIT_FUNC PyInit__serving(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "source_hash", KQ_SOURCE_HASH) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
