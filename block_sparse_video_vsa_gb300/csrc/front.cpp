// Front of the cache calls for Python: the checks of a call's tensors, the
// tensors that it makes and the call itself, for calls on the current device
// and stream.  A cache call's kernels take from 3 us; through ctypes, with its
// arguments looked at one attribute at a time, a call took 18 to 24 us of the
// host, here 2.4 with its tensors given and 5 to 7 with those it makes.  What
// this front does not take as it is (other types, another device, a shape that
// does not fit) it leaves, by returning False, to the Python function, which
// says what is wrong; a status of the library comes back as a number.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "vsa.h"

namespace {

// Other Python threads go on while tensors are made and kernels launched.
struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

decltype(&vsa_cache_append) append_fn;
decltype(&vsa_cache_read) read_fn;
decltype(&vsa_cache_attn) attn_fn;
decltype(&vsa_cache_attn_workspace_bytes) workspace_fn;

// A contiguous tensor of `type` on CUDA device `dev`, or null.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || t.scalar_type() != type ||
        !t.is_contiguous())
        return nullptr;
    for (int64_t n : t.sizes())
        if (n > INT32_MAX) return nullptr;
    return &t;
}
// The same where None stands for none: false if it is neither.
bool optional(PyObject* o, at::ScalarType type, int dev, const at::Tensor*& t) {
    t = nullptr;
    return o == Py_None || (t = tensor(o, type, dev)) != nullptr;
}
template <class T>
T* data(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

struct Cache {
    vsa_cache c;
    int dev;
    cudaStream_t stream;
    at::Device device() const { return at::Device(at::kCUDA, (c10::DeviceIndex)dev); }
};
bool cache(PyObject* pool_o, PyObject* table_o, PyObject* lens_o, PyObject* scale_o, Cache& x) {
    if (!THPVariable_Check(pool_o)) return false;
    const at::Tensor& p = THPVariable_Unpack(pool_o);
    if (!p.defined() || !p.is_cuda()) return false;
    x.dev = (int)p.get_device();
    if (x.dev != (int)c10::cuda::current_device()) return false;
    const at::Tensor *pool = tensor(pool_o, at::kByte, x.dev), *table = tensor(table_o, at::kInt, x.dev),
                     *lens = tensor(lens_o, at::kInt, x.dev), *scale;
    if (!pool || !table || !lens || !optional(scale_o, at::kFloat, x.dev, scale)) return false;
    if (pool->dim() != 3 || (pool->size(2) != 72 * 64 && pool->size(2) != 72 * 128)) return false;
    if (table->dim() != 2 || lens->dim() != 1 || lens->size(0) != table->size(0)) return false;
    if (scale && (scale->dim() != 2 || scale->size(0) != 2 || scale->size(1) != pool->size(1))) return false;
    x.c.pages = (int32_t)pool->size(0);
    x.c.kv_heads = (int32_t)pool->size(1);
    x.c.D = (int32_t)(pool->size(2) / 72);
    x.c.B = (int32_t)table->size(0);
    x.c.width = (int32_t)table->size(1);
    x.c.pool = pool->data_ptr();
    x.c.table = data<int32_t>(table);
    x.c.kv_lens = data<int32_t>(lens);
    x.c.kv_scale = data<float>(scale);
    x.stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)x.dev).stream();
    return true;
}

bool rows(const at::Tensor* t, int64_t B, int64_t D) { return t->dim() == 4 && t->size(0) == B && t->size(3) == D; }
bool vector(const at::Tensor* t, int64_t n) { return t->dim() == 1 && t->size(0) == n; }

// `given`, or a new tensor of these sizes, which `*made` then holds.
const at::Tensor* given_or_new(const at::Tensor* given, at::IntArrayRef sizes, at::ScalarType type, const Cache& x,
                               at::Tensor* made) {
    if (given) return given;
    *made = at::empty(sizes, at::TensorOptions().dtype(type).device(x.device()));
    return made;
}
PyObject* result(PyObject* given, const at::Tensor& made) {
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}
PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* t = a && b ? PyTuple_New(2) : nullptr;
    if (!t) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

// append(pool, k, v, table, kv_lens, new_lens, rope, positions, interleaved, q, q_out, kv_scale)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 12 || !cache(a[0], a[3], a[4], a[11], x)) Py_RETURN_FALSE;
    const at::Tensor *k = tensor(a[1], at::kBFloat16, x.dev), *v = tensor(a[2], at::kBFloat16, x.dev);
    const at::Tensor *fresh, *rope, *positions, *q, *q_out;
    if (!k || !v || !optional(a[5], at::kInt, x.dev, fresh) || !optional(a[6], at::kFloat, x.dev, rope) ||
        !optional(a[7], at::kInt, x.dev, positions) || !optional(a[9], at::kBFloat16, x.dev, q) ||
        !optional(a[10], at::kBFloat16, x.dev, q_out))
        Py_RETURN_FALSE;
    if (!rows(k, x.c.B, x.c.D) || k->size(2) != x.c.kv_heads || v->sizes() != k->sizes()) Py_RETURN_FALSE;
    const int64_t S = k->size(1);
    if (fresh && !vector(fresh, x.c.B)) Py_RETURN_FALSE;
    if (rope && (rope->dim() != 2 || rope->size(0) == 0 || rope->size(1) == 0)) Py_RETURN_FALSE;
    if (positions && (positions->dim() != 2 || positions->size(0) != x.c.B || positions->size(1) != S)) Py_RETURN_FALSE;
    if (q ? !rows(q, x.c.B, x.c.D) || q->size(1) != S || (q_out && q_out->sizes() != q->sizes()) : q_out != nullptr)
        Py_RETURN_FALSE;
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0) return nullptr;
    at::Tensor made;
    vsa_status st;
    {
        NoGil no_gil;
        if (q) q_out = given_or_new(q_out, q->sizes(), at::kBFloat16, x, &made);
        st = append_fn(&x.c, data<void>(q), data<void>(k), data<void>(v), (int32_t)S, q ? (int32_t)q->size(2) : 0,
                       data<int32_t>(fresh), data<float>(rope), rope ? (int32_t)rope->size(0) : 0,
                       rope ? (int32_t)rope->size(1) : 0, interleaved, data<int32_t>(positions), data<void>(q_out),
                       x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    if (!q) Py_RETURN_NONE;
    return result(a[10], made);
    END_HANDLE_TH_ERRORS
}

// read(pool, table, kv_lens, S, kv_scale, k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 7 || !cache(a[0], a[1], a[2], a[4], x) || !PyLong_Check(a[3])) Py_RETURN_FALSE;
    const int64_t S = PyLong_AsLongLong(a[3]);
    if (S == -1 && PyErr_Occurred()) PyErr_Clear();
    const at::Tensor *k, *v;
    if (S <= 0 || S > INT32_MAX || !optional(a[5], at::kBFloat16, x.dev, k) || !optional(a[6], at::kBFloat16, x.dev, v))
        Py_RETURN_FALSE;
    const int64_t shape[4] = {x.c.B, S, x.c.kv_heads, x.c.D};
    const at::IntArrayRef sizes(shape, 4);
    if ((k && k->sizes() != sizes) || (v && v->sizes() != sizes)) Py_RETURN_FALSE;
    at::Tensor made_k, made_v;
    vsa_status st;
    {
        NoGil no_gil;
        k = given_or_new(k, sizes, at::kBFloat16, x, &made_k);
        v = given_or_new(v, sizes, at::kBFloat16, x, &made_v);
        st = read_fn(&x.c, (int32_t)S, data<void>(k), data<void>(v), x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    PyObject* first = result(a[5], made_k);
    return pair(first, result(a[6], made_v));
    END_HANDLE_TH_ERRORS
}

// attn(q, pool, table, kv_lens, q_lens, causal, page_sel, kv_scale, sm_scale, workspace, out, lse, want_lse)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 13 || !cache(a[1], a[2], a[3], a[7], x)) Py_RETURN_FALSE;
    const at::Tensor *q = tensor(a[0], at::kBFloat16, x.dev), *q_lens, *sel, *work, *out, *lse;
    if (!q || !optional(a[4], at::kInt, x.dev, q_lens) || !optional(a[6], at::kInt, x.dev, sel) ||
        !optional(a[9], at::kByte, x.dev, work) || !optional(a[10], at::kBFloat16, x.dev, out) ||
        !optional(a[11], at::kFloat, x.dev, lse))
        Py_RETURN_FALSE;
    if (!rows(q, x.c.B, x.c.D)) Py_RETURN_FALSE;
    const int64_t Sq = q->size(1), heads = q->size(2);
    if (heads == 0 || x.c.kv_heads == 0 || heads % x.c.kv_heads) Py_RETURN_FALSE;
    if (q_lens && !vector(q_lens, x.c.B)) Py_RETURN_FALSE;
    if (sel && (sel->dim() != 3 || sel->size(0) != x.c.B || sel->size(1) != x.c.kv_heads || sel->size(2) == 0))
        Py_RETURN_FALSE;
    if (out && out->sizes() != q->sizes()) Py_RETURN_FALSE;
    const int64_t shape[3] = {x.c.B, heads, Sq};
    if (lse && lse->sizes() != at::IntArrayRef(shape, 3)) Py_RETURN_FALSE;
    const int causal = PyObject_IsTrue(a[5]), want_lse = PyObject_IsTrue(a[12]);
    const double scale = PyFloat_AsDouble(a[8]);
    if (causal < 0 || want_lse < 0 || (scale == -1.0 && PyErr_Occurred())) return nullptr;
    const int64_t bytes = (int64_t)workspace_fn(x.c.kv_heads, x.c.D, (int32_t)Sq, (int32_t)heads);
    if (bytes == 0 || (work && work->numel() < bytes)) Py_RETURN_FALSE;
    at::Tensor made_work, made_out, made_lse;
    vsa_status st;
    {
        NoGil no_gil;
        work = given_or_new(work, {bytes}, at::kByte, x, &made_work);
        out = given_or_new(out, q->sizes(), at::kBFloat16, x, &made_out);
        if (want_lse) lse = given_or_new(lse, at::IntArrayRef(shape, 3), at::kFloat, x, &made_lse);
        st = attn_fn(&x.c, data<void>(q), (int32_t)Sq, (int32_t)heads, data<int32_t>(q_lens), causal, data<int32_t>(sel),
                     sel ? (int32_t)sel->size(2) : 0, (float)scale, data<void>(work), data<void>(out), data<float>(lse),
                     x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    PyObject* first = result(a[10], made_out);
    return pair(first, lse ? result(a[11], made_lse) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// bind(append, read, attn, workspace_bytes): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i] && PyErr_Occurred()) return nullptr;
    }
    append_fn = reinterpret_cast<decltype(append_fn)>(p[0]);
    read_fn = reinterpret_cast<decltype(read_fn)>(p[1]);
    attn_fn = reinterpret_cast<decltype(attn_fn)>(p[2]);
    workspace_fn = reinterpret_cast<decltype(workspace_fn)>(p[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&module); }
