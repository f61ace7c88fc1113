// Front of the cache calls for Python: the checks of a call's tensors, the
// tensors that it makes and the call itself, for calls on the current device
// and stream.  A cache call's kernels take from 3 us; through ctypes, with its
// arguments looked at one attribute at a time, a call took 18 to 24 us of the
// host, here 2.2 with its tensors given and 3 to 7 with those it makes.  What
// this front does not take as it is (other types, another device, a shape that
// does not fit) it leaves, by returning False, to the Python function, which
// says what is wrong; a status of the library comes back as a number.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
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
decltype(&vsa_cache_attn_tree) attn_tree_fn;
decltype(&vsa_cache_tree) tree_fn;
decltype(&vsa_cache_accept) accept_fn;
decltype(&vsa_cache_weigh) weigh_fn;
decltype(&vsa_cache_evict) evict_fn;

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
    *made = at::detail::empty_cuda(sizes, type, x.device(), std::nullopt);  // (past the dispatcher: 0.5 us less)
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

// attn(q, pool, table, kv_lens, q_lens, causal, page_sel, kv_scale, sm_scale, workspace, out, lse, want_lse, tree)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 14 || !cache(a[1], a[2], a[3], a[7], x)) Py_RETURN_FALSE;
    const at::Tensor *q = tensor(a[0], at::kBFloat16, x.dev), *q_lens, *sel, *work, *out, *lse, *tree;
    if (!q || !optional(a[4], at::kInt, x.dev, q_lens) || !optional(a[6], at::kInt, x.dev, sel) ||
        !optional(a[9], at::kByte, x.dev, work) || !optional(a[10], at::kBFloat16, x.dev, out) ||
        !optional(a[11], at::kFloat, x.dev, lse) || !optional(a[13], at::kLong, x.dev, tree))
        Py_RETURN_FALSE;
    if (!rows(q, x.c.B, x.c.D)) Py_RETURN_FALSE;
    const int64_t Sq = q->size(1), heads = q->size(2);
    if (heads == 0 || x.c.kv_heads == 0 || heads % x.c.kv_heads) Py_RETURN_FALSE;
    if (q_lens && !vector(q_lens, x.c.B)) Py_RETURN_FALSE;
    if (sel && (sel->dim() != 3 || sel->size(0) != x.c.B || sel->size(1) != x.c.kv_heads || sel->size(2) == 0))
        Py_RETURN_FALSE;
    if (tree && (tree->dim() != 3 || tree->size(0) != x.c.B || tree->size(1) != Sq || tree->size(2) != (Sq + 63) / 64))
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
        const int32_t nsel = sel ? (int32_t)sel->size(2) : 0;
        if (tree)
            st = attn_tree_fn(&x.c, data<void>(q), (int32_t)Sq, (int32_t)heads, data<int32_t>(q_lens),
                              data<uint64_t>(tree), data<int32_t>(sel), nsel, (float)scale, data<void>(work),
                              data<void>(out), data<float>(lse), x.stream);
        else
            st = attn_fn(&x.c, data<void>(q), (int32_t)Sq, (int32_t)heads, data<int32_t>(q_lens), causal,
                         data<int32_t>(sel), nsel, (float)scale, data<void>(work), data<void>(out), data<float>(lse),
                         x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    PyObject* first = result(a[10], made_out);
    return pair(first, lse ? result(a[11], made_lse) : Py_NewRef(Py_None));
    END_HANDLE_TH_ERRORS
}

// tree(parents, kv_lens, new_lens, starts, mask, positions)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6 || !THPVariable_Check(a[0])) Py_RETURN_FALSE;
    const at::Tensor& p = THPVariable_Unpack(a[0]);
    if (!p.defined() || !p.is_cuda()) Py_RETURN_FALSE;
    Cache x;
    x.dev = (int)p.get_device();
    if (x.dev != (int)c10::cuda::current_device()) Py_RETURN_FALSE;
    const at::Tensor *parents = tensor(a[0], at::kInt, x.dev), *lens, *fresh, *starts, *mask, *positions;
    if (!parents || parents->dim() != 2 || !optional(a[1], at::kInt, x.dev, lens) ||
        !optional(a[2], at::kInt, x.dev, fresh) || !optional(a[3], at::kInt, x.dev, starts) ||
        !optional(a[4], at::kLong, x.dev, mask) || !optional(a[5], at::kInt, x.dev, positions))
        Py_RETURN_FALSE;
    const int64_t B = parents->size(0), S = parents->size(1);
    if ((lens && !vector(lens, B)) || (fresh && !vector(fresh, B)) || (starts && !vector(starts, B))) Py_RETURN_FALSE;
    const int64_t shape[3] = {B, S, (S + 63) / 64};
    if ((mask && mask->sizes() != at::IntArrayRef(shape, 3)) || (positions && positions->sizes() != parents->sizes()))
        Py_RETURN_FALSE;
    at::Tensor made_mask, made_positions;
    vsa_status st;
    {
        NoGil no_gil;
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)x.dev).stream();
        mask = given_or_new(mask, at::IntArrayRef(shape, 3), at::kLong, x, &made_mask);
        positions = given_or_new(positions, parents->sizes(), at::kInt, x, &made_positions);
        st = tree_fn(data<int32_t>(parents), (int32_t)B, (int32_t)S, data<int32_t>(lens), data<int32_t>(fresh),
                     data<int32_t>(starts), data<uint64_t>(mask), data<int32_t>(positions), stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    PyObject* first = result(a[4], made_mask);
    return pair(first, result(a[5], made_positions));
    END_HANDLE_TH_ERRORS
}

// accept(pool, table, kv_lens, new_lens, path, path_lens, lens)
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 7 || !cache(a[0], a[1], a[2], Py_None, x)) Py_RETURN_FALSE;
    const at::Tensor *fresh = tensor(a[3], at::kInt, x.dev), *path = tensor(a[4], at::kInt, x.dev),
                     *path_lens = tensor(a[5], at::kInt, x.dev), *lens;
    if (!fresh || !path || !path_lens || !optional(a[6], at::kInt, x.dev, lens)) Py_RETURN_FALSE;
    if (!vector(fresh, x.c.B) || !vector(path_lens, x.c.B) || path->dim() != 2 || path->size(0) != x.c.B ||
        (lens && !vector(lens, x.c.B)))
        Py_RETURN_FALSE;
    at::Tensor made;
    vsa_status st;
    {
        NoGil no_gil;
        lens = given_or_new(lens, {x.c.B}, at::kInt, x, &made);
        st = accept_fn(&x.c, data<int32_t>(fresh), data<int32_t>(path), data<int32_t>(path_lens),
                       (int32_t)path->size(1), data<int32_t>(lens), x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    return result(a[6], made);
    END_HANDLE_TH_ERRORS
}

// weigh(q, lse, pool, table, kv_lens, q_lens, causal, weights, out, kv_scale, sm_scale); out: None is a new tensor
PyObject* weigh(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 11 || !cache(a[2], a[3], a[4], a[9], x)) Py_RETURN_FALSE;
    const at::Tensor *q = tensor(a[0], at::kBFloat16, x.dev), *lse = tensor(a[1], at::kFloat, x.dev), *q_lens, *before,
                     *out;
    if (!q || !lse || !optional(a[5], at::kInt, x.dev, q_lens) || !optional(a[7], at::kFloat, x.dev, before) ||
        !optional(a[8], at::kFloat, x.dev, out))
        Py_RETURN_FALSE;
    if (!rows(q, x.c.B, x.c.D)) Py_RETURN_FALSE;
    const int64_t Sq = q->size(1), heads = q->size(2);
    if (heads == 0 || x.c.kv_heads == 0 || heads % x.c.kv_heads) Py_RETURN_FALSE;
    const int64_t sums[3] = {x.c.B, heads, Sq}, places[3] = {x.c.B, x.c.kv_heads, (int64_t)x.c.width * 64};
    if (lse->sizes() != at::IntArrayRef(sums, 3) || (q_lens && !vector(q_lens, x.c.B))) Py_RETURN_FALSE;
    if ((before && before->sizes() != at::IntArrayRef(places, 3)) || (out && out->sizes() != at::IntArrayRef(places, 3)))
        Py_RETURN_FALSE;
    const int causal = PyObject_IsTrue(a[6]);
    const double scale = PyFloat_AsDouble(a[10]);
    if (causal < 0 || (scale == -1.0 && PyErr_Occurred())) return nullptr;
    at::Tensor made;
    vsa_status st;
    {
        NoGil no_gil;
        out = given_or_new(out, at::IntArrayRef(places, 3), at::kFloat, x, &made);
        st = weigh_fn(&x.c, data<void>(q), data<float>(lse), (int32_t)Sq, (int32_t)heads, data<int32_t>(q_lens), causal,
                      (float)scale, data<float>(before), data<float>(out), x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    return result(a[8], made);
    END_HANDLE_TH_ERRORS
}

// evict(pool, table, kv_lens, weights, budget, first, recent, to_table, kept, lens, moved)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache x;
    if (n != 11 || !cache(a[0], a[1], a[2], Py_None, x)) Py_RETURN_FALSE;
    const at::Tensor *weights = tensor(a[3], at::kFloat, x.dev), *to, *kept, *lens, *moved;
    if (!weights || !optional(a[7], at::kInt, x.dev, to) || !optional(a[8], at::kInt, x.dev, kept) ||
        !optional(a[9], at::kInt, x.dev, lens) || !optional(a[10], at::kFloat, x.dev, moved))
        Py_RETURN_FALSE;
    int64_t sizes[3];
    for (int i = 0; i < 3; ++i) {
        if (!PyLong_Check(a[4 + i])) Py_RETURN_FALSE;
        sizes[i] = PyLong_AsLongLong(a[4 + i]);
        if (sizes[i] == -1 && PyErr_Occurred()) PyErr_Clear();
        if (sizes[i] < 0 || sizes[i] > INT32_MAX) Py_RETURN_FALSE;
    }
    const int64_t places[3] = {x.c.B, x.c.kv_heads, (int64_t)x.c.width * 64}, chosen[3] = {x.c.B, x.c.kv_heads, sizes[0]};
    if (sizes[0] == 0 || sizes[1] + sizes[2] > sizes[0]) Py_RETURN_FALSE;
    if (weights->sizes() != at::IntArrayRef(places, 3)) Py_RETURN_FALSE;
    if (to ? to->dim() != 2 || to->size(0) != x.c.B || to->size(1) == 0 : moved != nullptr) Py_RETURN_FALSE;
    const int64_t width = to ? to->size(1) : 0, after[3] = {x.c.B, x.c.kv_heads, width * 64};
    if ((kept && kept->sizes() != at::IntArrayRef(chosen, 3)) || (lens && !vector(lens, x.c.B)) ||
        (moved && moved->sizes() != at::IntArrayRef(after, 3)))
        Py_RETURN_FALSE;
    at::Tensor made_kept, made_lens, made_moved;
    vsa_status st;
    {
        NoGil no_gil;
        kept = given_or_new(kept, at::IntArrayRef(chosen, 3), at::kInt, x, &made_kept);
        lens = given_or_new(lens, {x.c.B}, at::kInt, x, &made_lens);
        if (to) moved = given_or_new(moved, at::IntArrayRef(after, 3), at::kFloat, x, &made_moved);
        st = evict_fn(&x.c, data<float>(weights), (int32_t)sizes[0], (int32_t)sizes[1], (int32_t)sizes[2],
                      data<int32_t>(to), (int32_t)width, data<int32_t>(kept), data<int32_t>(lens), data<float>(moved),
                      x.stream);
    }
    if (st != VSA_OK) return PyLong_FromLong(st);
    PyObject* t = PyTuple_New(3);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, result(a[9], made_lens));
    PyTuple_SET_ITEM(t, 1, result(a[8], made_kept));
    PyTuple_SET_ITEM(t, 2, to ? result(a[10], made_moved) : Py_NewRef(a[3]));
    for (int i = 0; i < 3; ++i)
        if (!PyTuple_GET_ITEM(t, i)) {
            Py_DECREF(t);
            return nullptr;
        }
    return t;
    END_HANDLE_TH_ERRORS
}

// bind(append, read, attn, workspace_bytes, attn_tree, tree, accept, weigh, evict): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr int kAddresses = 9;
    if (n != kAddresses) {
        PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
        return nullptr;
    }
    void* p[kAddresses];
    for (int i = 0; i < kAddresses; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i] && PyErr_Occurred()) return nullptr;
    }
    append_fn = reinterpret_cast<decltype(append_fn)>(p[0]);
    read_fn = reinterpret_cast<decltype(read_fn)>(p[1]);
    attn_fn = reinterpret_cast<decltype(attn_fn)>(p[2]);
    workspace_fn = reinterpret_cast<decltype(workspace_fn)>(p[3]);
    attn_tree_fn = reinterpret_cast<decltype(attn_tree_fn)>(p[4]);
    tree_fn = reinterpret_cast<decltype(tree_fn)>(p[5]);
    accept_fn = reinterpret_cast<decltype(accept_fn)>(p[6]);
    weigh_fn = reinterpret_cast<decltype(weigh_fn)>(p[7]);
    evict_fn = reinterpret_cast<decltype(evict_fn)>(p[8]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree)), METH_FASTCALL, nullptr},
    {"accept", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(accept)), METH_FASTCALL, nullptr},
    {"weigh", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(weigh)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&module); }
