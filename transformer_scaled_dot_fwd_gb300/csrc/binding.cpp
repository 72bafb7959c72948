// Python's usual calls of the serving entry points (attn_fwd_packed, attn_rope,
// attn_rope_append, attn_decode_tree), from tensors to the C ABI in one crossing:
// outputs are made here and the workspace comes from torch's caching allocator.
// The usual call is one whose arguments are all in order: plain strided tensors on
// the current device.  For any other a function returns None, and the package's
// checked path in Python takes the call, refuses it with its reason or runs it on
// the stream it names.  Nothing here computes, and nothing is kept between calls.
//
// What bounds such a call is the host (Grace): reading attributes, making an
// output and a workspace through Python's interpreter costs 11-14 us beside the
// library's own 4-6 us.  A rope call takes 5 us here against 17, a packed one 8-11
// against 22, a tree one 10-12 against 20.
#include <Python.h>

#include <cmath>
#include <climits>
#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

// the library's functions, as the package loaded them
decltype(&attn_fwd_packed) f_packed;
decltype(&attn_fwd_packed_workspace) f_packed_workspace;
decltype(&attn_rope) f_rope;
decltype(&attn_rope_append) f_rope_append;
decltype(&attn_decode_tree) f_tree;
decltype(&attn_decode_tree_workspace) f_tree_workspace;

bool small(int64_t n) { return n >= 0 && n <= INT_MAX; }

// A plain CUDA tensor's C++ side; null for anything else.
const at::Tensor* cuda_tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.defined() && t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

// What a call's tensors share.
struct Call {
    at::ScalarType dtype;
    at::Device device = at::kCPU;
    int code;

    // Takes them from q, a tensor of n dimensions on the current device.
    bool of(const at::Tensor* q, int n) {
        if (!q || q->dim() != n || q->stride(n - 1) != 1) return false;
        dtype = q->scalar_type();
        device = q->device();
        code = dtype == at::kBFloat16 ? ATTN_BF16 : ATTN_F32;
        if (dtype != at::kBFloat16 && dtype != at::kFloat) return false;
        for (int64_t s : q->sizes())
            if (!small(s)) return false;
        return device.index() == c10::cuda::current_device();
    }

    bool shares(const at::Tensor* t) const {
        return t && t->scalar_type() == dtype && t->device() == device;
    }

    // (T, heads, D) with contiguous head rows; its strides go to st.
    bool rows(const at::Tensor* t, int64_t T, int64_t D, long long* st) const {
        if (!shares(t) || t->dim() != 3 || t->size(0) != T || t->size(2) != D || t->stride(2) != 1 || !small(t->size(1)))
            return false;
        st[0] = t->stride(0), st[1] = t->stride(1);
        return true;
    }

    // A pair of contiguous (B, H_kv, Skv, D) caches.
    bool caches(const at::Tensor* k, const at::Tensor* v, int64_t D) const {
        if (!shares(k) || !shares(v) || k->dim() != 4 || k->sizes() != v->sizes() || k->size(3) != D) return false;
        for (int64_t s : k->sizes())
            if (!small(s)) return false;
        return k->is_contiguous() && v->is_contiguous();
    }

    // An int32 tensor of the given shape, or None.
    bool ints(PyObject* o, std::initializer_list<int64_t> shape, const int** p) const {
        *p = nullptr;
        if (o == Py_None) return true;
        const at::Tensor* t = cuda_tensor(o);
        if (!t || t->scalar_type() != at::kInt || t->device() != device || t->sizes() != at::IntArrayRef(shape) ||
            !t->is_contiguous())
            return false;
        *p = static_cast<const int*>(t->data_ptr());
        return true;
    }

    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    }
};

// An output: the caller's tensor, or one made here.
struct Out {
    PyObject* given = nullptr;
    at::Tensor made;
    const at::Tensor* t = nullptr;

    bool rows(PyObject* o, const Call& c, int64_t T, int64_t heads, int64_t D, long long* st) {
        if (o == Py_None) {
            made = c.make({T, heads, D}, c.dtype);
            t = &made;
            st[0] = heads * D, st[1] = D;
            return true;
        }
        given = o;
        t = cuda_tensor(o);
        return c.rows(t, T, D, st) && t->size(1) == heads;
    }
    void* ptr() const { return t ? t->data_ptr() : nullptr; }
    PyObject* object() {
        if (given) {
            Py_INCREF(given);
            return given;
        }
        return THPVariable_Wrap(std::move(made));
    }
};

bool frequencies(PyObject* o, int64_t D, const double** p, int* rotary_dim) {
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.device().is_cpu() || t.layout() != at::kStrided || t.scalar_type() != at::kDouble || t.dim() != 1 ||
        !t.is_contiguous() || 2 * t.size(0) > D)
        return false;
    *p = static_cast<const double*>(t.data_ptr());
    *rotary_dim = static_cast<int>(2 * t.size(0));
    return true;
}

// A Python float or int; None gives `otherwise` where that is a number.
bool number(PyObject* o, double otherwise, float* x) {
    if (o == Py_None && !std::isnan(otherwise)) {
        *x = static_cast<float>(otherwise);
        return true;
    }
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return false;
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *x = static_cast<float>(d);
    return true;
}

bool flag(PyObject* o, int* x) {
    if (!PyBool_Check(o)) return false;
    *x = o == Py_True;
    return true;
}

// Device memory for one call: given back when the call is enqueued, as the
// allocator reuses it in stream order.
struct Workspace {
    void* p = nullptr;
    Workspace(long long bytes, cudaStream_t stream) {
        if (bytes > 0) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(static_cast<size_t>(bytes), stream);
    }
    Workspace(const Workspace&) = delete;
    ~Workspace() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

// A launch may wait for room in the stream's queue: not with the interpreter locked.
template <class F>
int unlocked(F&& f) {
    PyThreadState* state = PyEval_SaveThread();
    const int rc = f();
    PyEval_RestoreThread(state);
    return rc;
}

PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* r = a && b ? PyTuple_New(2) : nullptr;
    if (!r) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        return nullptr;
    }
    PyTuple_SET_ITEM(r, 0, a);
    PyTuple_SET_ITEM(r, 1, b);
    return r;
}

const double kNone = std::nan("");

// packed(q, k, v, cu_seqlens, out, lse, scale, causal, return_lse)
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v;
    Call c;
    long long st[8];
    if (n != 9 || !(q = cuda_tensor(a[0])) || !c.of(q, 3) || !(k = cuda_tensor(a[1])) || !(v = cuda_tensor(a[2])))
        Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    if (!c.rows(k, T, D, st + 2) || !c.rows(v, T, D, st + 4)) Py_RETURN_NONE;
    const int64_t H_kv = k->size(1);
    const at::Tensor* cu = cuda_tensor(a[3]);
    if (v->size(1) != H_kv || H_kv < 1 || H % H_kv || D < 1 || !cu || cu->dim() != 1 || cu->size(0) < 1 ||
        !small(cu->size(0)))
        Py_RETURN_NONE;
    const int n_seq = static_cast<int>(cu->size(0) - 1);
    const int* cu_p;
    float scale;
    int causal, want_lse;
    if (!c.ints(a[3], {n_seq + 1}, &cu_p) || !number(a[6], 1.0 / std::sqrt(static_cast<double>(D)), &scale) ||
        !flag(a[7], &causal) || !flag(a[8], &want_lse))
        Py_RETURN_NONE;
    Out lse;
    if (a[5] != Py_None) {
        lse.given = a[5];
        lse.t = cuda_tensor(a[5]);
        if (!lse.t || lse.t->scalar_type() != at::kFloat || lse.t->sizes() != at::IntArrayRef({T, H}) ||
            !lse.t->is_contiguous() || lse.t->device() != c.device)
            Py_RETURN_NONE;
    }
    Out out;
    if (!out.rows(a[4], c, T, H, D, st + 6)) Py_RETURN_NONE;
    if (a[5] == Py_None && want_lse) {
        lse.made = c.make({T, H}, at::kFloat);
        lse.t = &lse.made;
    }
    const long long need = f_packed_workspace(T, n_seq, H, H_kv, c.code);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    Workspace ws(need, stream);
    const int rc = unlocked([&] {
        return f_packed(q->data_ptr(), k->data_ptr(), v->data_ptr(), out.ptr(), static_cast<float*>(lse.ptr()), T, H, H_kv,
                        D, st, cu_p, n_seq, scale, causal, c.code, ws.p, need, stream);
    });
    if (rc) Py_RETURN_NONE;
    return lse.t ? pair(out.object(), lse.object()) : out.object();
    END_HANDLE_TH_ERRORS
}

// rope(q, k, positions, freqs, q_out, k_out, interleaved, inverse, mscale)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k = nullptr;
    Call c;
    long long st[8] = {};
    if (n != 9 || !(q = cuda_tensor(a[0])) || !c.of(q, 3)) Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    const int* pos;
    const double* freqs;
    int rotary_dim, interleaved, inverse;
    float mscale;
    if (a[2] == Py_None || !c.ints(a[2], {T}, &pos) || !frequencies(a[3], D, &freqs, &rotary_dim) ||
        !flag(a[6], &interleaved) || !flag(a[7], &inverse) || !number(a[8], kNone, &mscale))
        Py_RETURN_NONE;
    int64_t H_kv = 0;
    if (a[1] != Py_None) {
        k = cuda_tensor(a[1]);
        if (!c.rows(k, T, D, st + 2)) Py_RETURN_NONE;
        H_kv = k->size(1);
    } else if (a[5] != Py_None) {
        Py_RETURN_NONE;
    }
    Out q_out, k_out;
    if (!q_out.rows(a[4], c, T, H, D, st + 4) || (k && !k_out.rows(a[5], c, T, H_kv, D, st + 6))) Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    const int rc = unlocked([&] {
        return f_rope(q->data_ptr(), k ? k->data_ptr() : nullptr, q_out.ptr(), k_out.ptr(), T, H, H_kv, D, st, pos, freqs,
                      rotary_dim, interleaved, inverse, mscale, c.code, stream);
    });
    if (rc) Py_RETURN_NONE;
    return k ? pair(q_out.object(), k_out.object()) : q_out.object();
    END_HANDLE_TH_ERRORS
}

// rope_append(q, k, v, kcache, vcache, freqs, cu_seqlens, cache_len, positions, q_out, k_out, interleaved, mscale)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v, *kc, *vc;
    Call c;
    long long st[10] = {};
    if (n != 13 || !(q = cuda_tensor(a[0])) || !c.of(q, 3) || !(k = cuda_tensor(a[1])) || !(v = cuda_tensor(a[2])) ||
        !(kc = cuda_tensor(a[3])) || !(vc = cuda_tensor(a[4])))
        Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    if (!c.rows(k, T, D, st + 2) || !c.rows(v, T, D, st + 4) || !c.caches(kc, vc, D)) Py_RETURN_NONE;
    const int64_t H_kv = k->size(1), B = kc->size(0), Skv = kc->size(2);
    const int *cu, *cache_len, *pos;
    const double* freqs;
    int rotary_dim, interleaved;
    float mscale;
    if (v->size(1) != H_kv || kc->size(1) != H_kv || !frequencies(a[5], D, &freqs, &rotary_dim) ||
        !c.ints(a[6], {B + 1}, &cu) || !c.ints(a[7], {B}, &cache_len) || !c.ints(a[8], {T}, &pos) ||
        !flag(a[11], &interleaved) || !number(a[12], kNone, &mscale))
        Py_RETURN_NONE;
    Out q_out, k_out;
    const bool turned = a[10] != Py_None;
    if (!q_out.rows(a[9], c, T, H, D, st + 6) || (turned && !k_out.rows(a[10], c, T, H_kv, D, st + 8))) Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    const int rc = unlocked([&] {
        return f_rope_append(q->data_ptr(), k->data_ptr(), v->data_ptr(), q_out.ptr(), k_out.ptr(), kc->data_ptr(),
                             vc->data_ptr(), T, H, H_kv, D, st, B, Skv, cu, cache_len, pos, freqs, rotary_dim,
                             interleaved, mscale, c.code, stream);
    });
    if (rc) Py_RETURN_NONE;
    return turned ? pair(q_out.object(), k_out.object()) : q_out.object();
    END_HANDLE_TH_ERRORS
}

// tree(q, kcache, vcache, parents, cache_len, draft_len, out, scale)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *kc, *vc, *parents;
    Call c;
    if (n != 8 || !(q = cuda_tensor(a[0])) || !c.of(q, 4) || !(kc = cuda_tensor(a[1])) || !(vc = cuda_tensor(a[2])) ||
        !(parents = cuda_tensor(a[3])))
        Py_RETURN_NONE;
    const int64_t B = q->size(0), H = q->size(1), T = q->size(2), D = q->size(3);
    if (!c.caches(kc, vc, D)) Py_RETURN_NONE;
    const int64_t H_kv = kc->size(1), Skv = kc->size(2);
    const bool one = parents->dim() == 1;
    const int *par, *cache_len, *draft_len;
    float scale;
    if (kc->size(0) != B || H_kv < 1 || H % H_kv || D < 1 ||
        !(one ? c.ints(a[3], {T}, &par) : c.ints(a[3], {B, T}, &par)) || !c.ints(a[4], {B}, &cache_len) ||
        !c.ints(a[5], {B}, &draft_len) || !number(a[7], 1.0 / std::sqrt(static_cast<double>(D)), &scale))
        Py_RETURN_NONE;
    Out out;
    if (a[6] == Py_None) {
        out.made = at::empty_like(*q);
        out.t = &out.made;
    } else {
        out.given = a[6];
        out.t = cuda_tensor(a[6]);
        if (!c.shares(out.t) || out.t->sizes() != q->sizes() || out.t->stride(3) != 1) Py_RETURN_NONE;
    }
    const long long st[6] = {q->stride(0), q->stride(1), q->stride(2), out.t->stride(0), out.t->stride(1), out.t->stride(2)};
    const long long need = B && T > 0 && T <= 128 ? f_tree_workspace(B, H, H_kv, T, Skv, D, c.code) : 0;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    Workspace ws(need, stream);
    const int rc = unlocked([&] {
        return f_tree(q->data_ptr(), kc->data_ptr(), vc->data_ptr(), out.ptr(), B, H, H_kv, T, Skv, D, st, par,
                      one ? 0 : static_cast<int>(T), cache_len, draft_len, scale, c.code, ws.p, need > 0 ? need : 0, stream);
    });
    if (rc) Py_RETURN_NONE;
    return out.object();
    END_HANDLE_TH_ERRORS
}

// bind(packed, packed_workspace, rope, rope_append, tree, tree_workspace): their addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[6];
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    f_packed = reinterpret_cast<decltype(f_packed)>(p[0]);
    f_packed_workspace = reinterpret_cast<decltype(f_packed_workspace)>(p[1]);
    f_rope = reinterpret_cast<decltype(f_rope)>(p[2]);
    f_rope_append = reinterpret_cast<decltype(f_rope_append)>(p[3]);
    f_tree = reinterpret_cast<decltype(f_tree)>(p[4]);
    f_tree_workspace = reinterpret_cast<decltype(f_tree_workspace)>(p[5]);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"packed", fast(packed), METH_FASTCALL, nullptr},
    {"rope", fast(rope), METH_FASTCALL, nullptr},
    {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
    {"tree", fast(tree), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
