// CPython module _paged_fast: checks and marshals the paged operators' tensors
// and calls the library, for paged.py.  A decode step makes these calls once a
// layer, and the same checks in Python cost 6 us a call, more than its launch.
//
// A function returns the library's status, or None where an argument is not what
// a call takes at once: paged.py then goes through its own checks, which accept
// the call or say what is wrong.  So nothing here raises, and every condition is
// at least as strict as the one there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gemv_paged.h"

namespace {

decltype(&gemv_paged_slots) call_slots;
decltype(&gemv_paged_append) call_append;
decltype(&gemv_paged_attn) call_attn;

constexpr auto kInt = at::kInt;

struct Args {
    PyObject *const *at;
    int64_t device; // the current GPU
    bool ok = true;

    // Tensor i, on the current GPU, of this type; a null tensor otherwise.
    const at::Tensor *tensor(int i)
    {
        if (!THPVariable_Check(at[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(at[i]);
        if (t.layout() != at::kStrided || !t.is_cuda() || t.device().index() != device) {
            ok = false;
            return nullptr;
        }
        return &t;
    }

    // Address of a contiguous tensor of n values (any number if n < 0) in one dimension.
    template <class T> T *row(int i, at::ScalarType type, int64_t n)
    {
        const at::Tensor *t = tensor(i);
        if (!t || t->scalar_type() != type || t->dim() != 1 || (n >= 0 && t->size(0) != n) || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return static_cast<T *>(t->data_ptr());
    }

    int64_t whole(int i)
    {
        const int64_t v = PyLong_Check(at[i]) ? PyLong_AsLongLong(at[i]) : -1;
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }

    void *address(int i) { return PyLong_Check(at[i]) ? PyLong_AsVoidPtr(at[i]) : (ok = false, nullptr); }
};

int type_code(at::ScalarType t)
{
    return t == at::kFloat ? GEMV_W_F32 : t == at::kHalf ? GEMV_W_F16 : t == at::kBFloat16 ? GEMV_W_BF16 : -1;
}

bool cache_of(Args &a, int i, gemv_kv_cache *c)
{
    const at::Tensor *k = a.tensor(i), *v = a.tensor(i + 1);
    if (!k || !v || k->dim() != 4 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() ||
        k->stride(3) != 1 || v->stride(3) != 1 || type_code(k->scalar_type()) < 1)
        return false;
    if (k->size(1) > INT32_MAX || k->size(2) > INT32_MAX || k->size(3) > INT32_MAX)
        return false;
    c->k = k->data_ptr();
    c->v = v->data_ptr();
    c->type = type_code(k->scalar_type());
    c->num_pages = k->size(0);
    c->page_size = (int32_t)k->size(1);
    c->heads = (int32_t)k->size(2);
    c->dim = (int32_t)k->size(3);
    for (int d = 0; d < 3; ++d) {
        c->k_stride[d] = k->stride(d);
        c->v_stride[d] = v->stride(d);
    }
    return true;
}

struct Table {
    int32_t *p;
    int64_t width, stride;
};

bool table_of(Args &a, int i, int64_t requests, Table *out)
{
    const at::Tensor *t = a.tensor(i);
    if (!t || t->scalar_type() != kInt || t->dim() != 2 || t->size(0) != requests || (t->stride(1) != 1 && t->size(1) > 1))
        return false;
    *out = Table{static_cast<int32_t *>(t->data_ptr()), t->size(1), t->stride(0)};
    return true;
}

// [tokens, heads, dim] whose heads lie together in a row.
const void *rows_of(Args &a, int i, at::ScalarType type, int64_t tokens, int64_t heads, int64_t dim, int64_t *stride)
{
    const at::Tensor *t = a.tensor(i);
    if (!t || t->scalar_type() != type || t->dim() != 3 || t->size(0) != tokens || t->size(1) != heads ||
        t->size(2) != dim || t->stride(2) != 1 || (heads > 1 && t->stride(1) != dim)) {
        a.ok = false;
        return nullptr;
    }
    *stride = t->stride(0);
    return t->data_ptr();
}

// A library call's status, with the interpreter free for other threads meanwhile: a
// launch waits where the stream's queue is full.  The caller holds the tensors.
template <class F> PyObject *answer(F call)
{
    PyThreadState *state = PyEval_SaveThread();
    const int status = call();
    PyEval_RestoreThread(state);
    return PyLong_FromLong(status);
}

PyObject *none() { Py_RETURN_NONE; }

// (cached, fresh, free_pages, page_size, block_table, query_start, kv_len, token_request, positions, slots, used,
//  device, stream)
PyObject *slots(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 13)
        return none();
    Args a{args, PyLong_AsLongLong(args[11])};
    const auto *cached = a.row<const int32_t>(0, kInt, -1);
    if (!a.ok)
        return none();
    const int64_t requests = THPVariable_Unpack(args[0]).size(0);
    const auto *fresh = a.row<const int32_t>(1, kInt, requests);
    const auto *free_pages = a.row<const int32_t>(2, kInt, -1);
    const int64_t page = a.whole(3);
    auto *query_start = a.row<int32_t>(5, kInt, requests + 1);
    auto *kv_len = a.row<int32_t>(6, kInt, requests);
    auto *map = a.row<int32_t>(9, kInt, -1);
    if (!a.ok)
        return none();
    const int64_t tokens = THPVariable_Unpack(args[9]).size(0);
    auto *request = a.row<int32_t>(7, kInt, tokens);
    auto *positions = a.row<int32_t>(8, kInt, tokens);
    auto *used = a.row<int32_t>(10, kInt, 1);
    void *stream = a.address(12);
    Table t;
    if (!a.ok || !table_of(a, 4, requests, &t))
        return none();
    const int64_t num_free = THPVariable_Unpack(args[2]).size(0);
    return answer([&] {
        return call_slots(cached, fresh, requests, free_pages, num_free, page, t.p, t.width, t.stride, tokens, query_start,
                          kv_len, request, positions, map, used, stream);
    });
}

// (q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, axis, style, device, stream)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 13)
        return none();
    Args a{args, PyLong_AsLongLong(args[11])};
    const at::Tensor *q = a.tensor(0), *out = a.tensor(6), *pos = a.tensor(3);
    gemv_kv_cache c;
    if (!a.ok || q->dim() != 3 || type_code(q->scalar_type()) < 0 || !cache_of(a, 7, &c) || q->size(2) != c.dim)
        return none();
    const int64_t tokens = q->size(0), q_heads = q->size(1);
    int64_t qs, ks, vs;
    const void *qp = rows_of(a, 0, q->scalar_type(), tokens, q_heads, c.dim, &qs);
    const void *kp = rows_of(a, 1, q->scalar_type(), tokens, c.heads, c.dim, &ks);
    const void *vp = rows_of(a, 2, q->scalar_type(), tokens, c.heads, c.dim, &vs);
    const int64_t axes = pos->dim() == 2 ? pos->size(0) : 1;
    if (pos->scalar_type() != kInt || pos->dim() < 1 || pos->dim() > 2 || pos->size(pos->dim() - 1) != tokens ||
        !pos->is_contiguous() || out->dim() != 3 || out->size(0) != tokens || out->size(1) != q_heads ||
        out->size(2) != c.dim || type_code(out->scalar_type()) != c.type || !out->is_contiguous())
        return none();
    const auto *inv = a.row<const float>(4, at::kFloat, -1);
    if (!a.ok)
        return none();
    const int64_t half = THPVariable_Unpack(args[4]).size(0);
    const auto *map = a.row<const int32_t>(5, kInt, tokens);
    const int32_t *axis = args[9] == Py_None ? nullptr : a.row<const int32_t>(9, kInt, half);
    const int64_t style = a.whole(10);
    void *stream = a.address(12);
    if (!a.ok || style > 1)
        return none();
    const int type = type_code(q->scalar_type());
    const auto *positions = static_cast<const int32_t *>(pos->data_ptr());
    void *q_out = out->data_ptr();
    return answer([&] {
        return call_append(qp, kp, vp, type, tokens, q_heads, qs, ks, vs, positions, axes, axis, inv, 2 * half, (int)style,
                           map, q_out, &c, stream);
    });
}

// (q, k_cache, v_cache, block_table, query_start, kv_len, scale, dst, workspace, window, sinks, device, stream)
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 13)
        return none();
    Args a{args, PyLong_AsLongLong(args[11])};
    const at::Tensor *q = a.tensor(0), *dst = a.tensor(7), *work = args[8] == Py_None ? nullptr : a.tensor(8);
    gemv_kv_cache c;
    if (!a.ok || !cache_of(a, 1, &c) || q->dim() != 3 || type_code(q->scalar_type()) != c.type || q->size(2) != c.dim ||
        dst->sizes() != q->sizes() || type_code(dst->scalar_type()) < 0 || q->stride(2) != 1 || dst->stride(2) != 1 ||
        (work && !work->is_contiguous()) || !PyFloat_Check(args[6]))
        return none();
    const auto *kv_len = a.row<const int32_t>(5, kInt, -1);
    if (!a.ok)
        return none();
    const int64_t requests = THPVariable_Unpack(args[5]).size(0);
    const auto *query_start = a.row<const int32_t>(4, kInt, requests + 1);
    const int64_t window = a.whole(9), sinks = a.whole(10);
    void *stream = a.address(12);
    Table t;
    if (!a.ok || !table_of(a, 3, requests, &t))
        return none();
    const float scale = (float)PyFloat_AS_DOUBLE(args[6]);
    const void *qp = q->data_ptr();
    void *out = dst->data_ptr(), *scratch = work ? work->data_ptr() : nullptr;
    const int64_t qs[2] = {q->stride(0), q->stride(1)}, os[2] = {dst->stride(0), dst->stride(1)};
    const int64_t tokens = q->size(0), q_heads = q->size(1), bytes = work ? (int64_t)work->nbytes() : 0;
    const int type = type_code(dst->scalar_type());
    return answer([&] {
        return call_attn(qp, qs[0], qs[1], &c, t.p, t.width, t.stride, query_start, kv_len, requests, tokens, q_heads, scale,
                         window, sinks, out, type, os[0], os[1], scratch, bytes, stream);
    });
}

// (address of gemv_paged_slots, of gemv_paged_append, of gemv_paged_attn): the library that paged.py has loaded
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
        return nullptr;
    }
    call_slots = reinterpret_cast<decltype(call_slots)>(PyLong_AsVoidPtr(args[0]));
    call_append = reinterpret_cast<decltype(call_append)>(PyLong_AsVoidPtr(args[1]));
    call_attn = reinterpret_cast<decltype(call_attn)>(PyLong_AsVoidPtr(args[2]));
    if (PyErr_Occurred())
        return nullptr;
    return none();
}

// A C++ exception must not pass through C frames of the interpreter.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        PyObject *r = F(self, args, n);
        if (r && PyErr_Occurred()) // an integer that does not fit
            PyErr_Clear();
        return r;
    } catch (...) {
        PyErr_Clear();
        return none();
    }
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction entry()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef kMethods[] = {{"bind", entry<bind>(), METH_FASTCALL, nullptr},
                          {"slots", entry<slots>(), METH_FASTCALL, nullptr},
                          {"append", entry<append>(), METH_FASTCALL, nullptr},
                          {"attn", entry<attn>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged_fast", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__paged_fast() { return PyModule_Create(&kModule); }
