// Python's usual calls of the serving entry points (attn_fwd_packed, attn_rope,
// attn_rope_append, attn_decode_tree and those of a paged cache), from tensors to the C ABI in one crossing:
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
decltype(&attn_fwd_paged) f_paged;
decltype(&attn_fwd_paged_workspace) f_paged_workspace;
decltype(&attn_norm_rope) f_norm_rope;
decltype(&attn_rope_append_paged) f_append_paged;
decltype(&attn_pages_step) f_pages_step;
decltype(&attn_pages_compact) f_pages_compact;
decltype(&attn_pages_copy) f_pages_copy;
decltype(&attn_pages_workspace) f_pages_workspace;

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

    // A pair of (n_pages, H_kv, P, D) page pools with contiguous rows; their strides go to st.
    bool pages(const at::Tensor* k, const at::Tensor* v, int64_t D, long long* st) const {
        if (!shares(k) || !shares(v) || k->dim() != 4 || k->sizes() != v->sizes() || k->size(3) != D || k->stride(3) != 1 ||
            v->stride(3) != 1)
            return false;
        for (int64_t s : k->sizes())
            if (!small(s)) return false;
        for (int i = 0; i < 3; ++i) st[i] = k->stride(i), st[3 + i] = v->stride(i);
        return true;
    }

    // A (rows, entries) int32 table with contiguous rows.
    bool table(const at::Tensor* t) const {
        return t && t->scalar_type() == at::kInt && t->device() == device && t->dim() == 2 && t->stride(1) == 1 &&
               small(t->size(0)) && small(t->size(1));
    }

    // A (D,) weight in the call's dtype, or None.
    bool weight(PyObject* o, int64_t D, const void** p) const {
        *p = nullptr;
        if (o == Py_None) return true;
        const at::Tensor* t = cuda_tensor(o);
        if (!shares(t) || t->dim() != 1 || t->size(0) != D || !t->is_contiguous()) return false;
        *p = t->data_ptr();
        return true;
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

// A given (T, H) log-sum-exp, one made here, or none.
bool lse_of(PyObject* o, bool want, const Call& c, int64_t T, int64_t H, Out* lse) {
    if (o != Py_None) {
        lse->given = o;
        lse->t = cuda_tensor(o);
        return lse->t && lse->t->scalar_type() == at::kFloat && lse->t->sizes() == at::IntArrayRef({T, H}) &&
               lse->t->is_contiguous() && lse->t->device() == c.device;
    }
    if (want) {
        lse->made = c.make({T, H}, at::kFloat);
        lse->t = &lse->made;
    }
    return true;
}

// paged(q, kpages, vpages, page_table, cache_len, cu_seqlens, out, lse, scale, return_lse)
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *kp, *vp, *table;
    Call c;
    long long st[10];
    if (n != 10 || !(q = cuda_tensor(a[0])) || !c.of(q, 3) || !(kp = cuda_tensor(a[1])) || !(vp = cuda_tensor(a[2])) ||
        !(table = cuda_tensor(a[3])))
        Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    if (!c.pages(kp, vp, D, st + 4) || !c.table(table)) Py_RETURN_NONE;
    const int64_t n_pages = kp->size(0), H_kv = kp->size(1), P = kp->size(2), n_seq = table->size(0), M = table->size(1);
    const int *cu, *cache_len;
    float scale;
    int want_lse;
    if (H_kv < 1 || H % H_kv || D < 1 || !c.ints(a[4], {n_seq}, &cache_len) || !c.ints(a[5], {n_seq + 1}, &cu) ||
        (!cu && (n_seq == 0 || T % n_seq)) || !number(a[8], 1.0 / std::sqrt(static_cast<double>(D)), &scale) ||
        !flag(a[9], &want_lse))
        Py_RETURN_NONE;
    const long long need = f_paged_workspace(T, n_seq, H, H_kv, D, M, P, cu != nullptr, c.code);
    if (need < 0) Py_RETURN_NONE;
    Out lse, out;
    if (!out.rows(a[6], c, T, H, D, st + 2) || !lse_of(a[7], want_lse, c, T, H, &lse)) Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    Workspace ws(need, stream);
    const int rc = unlocked([&] {
        return f_paged(q->data_ptr(), kp->data_ptr(), vp->data_ptr(), out.ptr(), static_cast<float*>(lse.ptr()), T, H, H_kv, D,
                       st, n_pages, P, static_cast<const int*>(table->data_ptr()), M, table->stride(0), cu, cache_len, n_seq,
                       scale, c.code, ws.p, need, stream);
    });
    if (rc) Py_RETURN_NONE;
    return lse.t ? pair(out.object(), lse.object()) : out.object();
    END_HANDLE_TH_ERRORS
}

// norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, q_out, k_out, interleaved, mscale)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k = nullptr;
    Call c;
    long long st[8] = {};
    if (n != 11 || !(q = cuda_tensor(a[0])) || !c.of(q, 3)) Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    const int* pos;
    const double* freqs;
    const void *wq, *wk;
    int rotary_dim, interleaved;
    float eps, mscale;
    if (a[2] == Py_None || !c.ints(a[2], {T}, &pos) || !frequencies(a[3], D, &freqs, &rotary_dim) ||
        !c.weight(a[4], D, &wq) || !c.weight(a[5], D, &wk) || !number(a[6], kNone, &eps) || !flag(a[9], &interleaved) ||
        !number(a[10], kNone, &mscale))
        Py_RETURN_NONE;
    int64_t H_kv = 0;
    if (a[1] != Py_None) {
        k = cuda_tensor(a[1]);
        if (!c.rows(k, T, D, st + 2)) Py_RETURN_NONE;
        H_kv = k->size(1);
    } else if (a[8] != Py_None || a[5] != Py_None) {
        Py_RETURN_NONE;
    }
    Out q_out, k_out;
    if (!q_out.rows(a[7], c, T, H, D, st + 4) || (k && !k_out.rows(a[8], c, T, H_kv, D, st + 6))) Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    const int rc = unlocked([&] {
        return f_norm_rope(q->data_ptr(), k ? k->data_ptr() : nullptr, q_out.ptr(), k_out.ptr(), T, H, H_kv, D, st, pos, freqs,
                           rotary_dim, interleaved, mscale, wq, wk, eps, c.code, stream);
    });
    if (rc) Py_RETURN_NONE;
    return k ? pair(q_out.object(), k_out.object()) : q_out.object();
    END_HANDLE_TH_ERRORS
}

// append_paged(q, k, v, kpages, vpages, page_table, freqs, cache_len, cu_seqlens, positions, q_weight, k_weight, eps,
//              q_out, k_out, interleaved, mscale)
PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v, *kp, *vp, *table;
    Call c;
    long long st[16] = {};
    if (n != 17 || !(q = cuda_tensor(a[0])) || !c.of(q, 3) || !(k = cuda_tensor(a[1])) || !(v = cuda_tensor(a[2])) ||
        !(kp = cuda_tensor(a[3])) || !(vp = cuda_tensor(a[4])) || !(table = cuda_tensor(a[5])))
        Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    st[0] = q->stride(0), st[1] = q->stride(1);
    if (!c.rows(k, T, D, st + 2) || !c.rows(v, T, D, st + 4) || !c.pages(kp, vp, D, st + 10) || !c.table(table)) Py_RETURN_NONE;
    const int64_t H_kv = k->size(1), n_pages = kp->size(0), P = kp->size(2), n_seq = table->size(0), M = table->size(1);
    const int *cu, *cache_len, *pos;
    const double* freqs;
    const void *wq, *wk;
    int rotary_dim, interleaved;
    float eps, mscale;
    if (v->size(1) != H_kv || kp->size(1) != H_kv || n_seq == 0 || !frequencies(a[6], D, &freqs, &rotary_dim) ||
        !c.ints(a[7], {n_seq}, &cache_len) || !c.ints(a[8], {n_seq + 1}, &cu) || !c.ints(a[9], {T}, &pos) ||
        !c.weight(a[10], D, &wq) || !c.weight(a[11], D, &wk) || !number(a[12], kNone, &eps) || !flag(a[15], &interleaved) ||
        !number(a[16], kNone, &mscale))
        Py_RETURN_NONE;
    Out q_out, k_out;
    const bool turned = a[14] != Py_None;
    if (!q_out.rows(a[13], c, T, H, D, st + 6) || (turned && !k_out.rows(a[14], c, T, H_kv, D, st + 8))) Py_RETURN_NONE;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    const int rc = unlocked([&] {
        return f_append_paged(q->data_ptr(), k->data_ptr(), v->data_ptr(), q_out.ptr(), k_out.ptr(), kp->data_ptr(),
                              vp->data_ptr(), T, H, H_kv, D, st, n_pages, P, static_cast<const int*>(table->data_ptr()), M,
                              table->stride(0), cu, cache_len, n_seq, pos, freqs, rotary_dim, interleaved, mscale, wq, wk, eps,
                              c.code, stream);
    });
    if (rc) Py_RETURN_NONE;
    return turned ? pair(q_out.object(), k_out.object()) : q_out.object();
    END_HANDLE_TH_ERRORS
}

// A Python int that fits 32 bits.
bool whole(PyObject* o, int64_t* x) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    *x = PyLong_AsLongLongAndOverflow(o, &overflow);
    return !overflow && small(*x);
}

// int32 outputs, made here: the usual call gives none.
template <size_t N>
PyObject* tuple_of(at::Tensor (&t)[N]) {
    PyObject* r = PyTuple_New(N);
    for (size_t i = 0; r && i < N; ++i) {
        PyObject* o = THPVariable_Wrap(std::move(t[i]));
        if (!o) Py_CLEAR(r);
        else PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

// A table on the current device, as the first argument of a call about pages.
bool first_table(PyObject* o, const at::Tensor** t, Call* c) {
    *t = cuda_tensor(o);
    if (!*t) return false;
    c->device = (*t)->device();
    return c->device.index() == c10::cuda::current_device() && c->table(*t);
}

// pages_step(page_table, cache_len, n_pages, page_size, parents, new_len, pinned, out)
PyObject* pages_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* table;
    Call c;
    int64_t n_pages, P;
    if (n != 8 || a[7] != Py_None || !first_table(a[0], &table, &c) || !whole(a[2], &n_pages) || !whole(a[3], &P)) Py_RETURN_NONE;
    const int64_t n_seq = table->size(0), M = table->size(1);
    int64_t n_out = n_seq;
    if (a[4] != Py_None) {
        const at::Tensor* p = cuda_tensor(a[4]);
        if (!p || p->dim() != 1 || !small(p->size(0))) Py_RETURN_NONE;
        n_out = p->size(0);
    }
    const int *cache_len, *parents, *new_len, *pinned;
    if (!c.ints(a[1], {n_seq}, &cache_len) || !c.ints(a[4], {n_out}, &parents) || !c.ints(a[5], {n_out}, &new_len) ||
        !c.ints(a[6], {n_pages}, &pinned))
        Py_RETURN_NONE;
    at::Tensor r[4] = {c.make({n_out, M}, at::kInt), c.make({n_out}, at::kInt), c.make({n_out, 3}, at::kInt), c.make({1}, at::kInt)};
    const long long need = f_pages_workspace(n_out, n_pages);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    Workspace ws(need, stream);
    int* o[4];
    for (int i = 0; i < 4; ++i) o[i] = static_cast<int*>(r[i].data_ptr());
    const int rc = unlocked([&] {
        return f_pages_step(static_cast<const int*>(table->data_ptr()), cache_len, n_seq, M, table->stride(0), n_pages, P,
                            parents, new_len, pinned, n_out, o[0], M, o[1], o[2], o[3], ws.p, need, stream);
    });
    if (rc) Py_RETURN_NONE;
    return tuple_of(r);
    END_HANDLE_TH_ERRORS
}

// pages_compact(page_table, cache_len, n_pages, page_size, pinned, out)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* table;
    Call c;
    int64_t n_pages, P;
    if (n != 6 || a[5] != Py_None || !first_table(a[0], &table, &c) || !whole(a[2], &n_pages) || !whole(a[3], &P)) Py_RETURN_NONE;
    const int64_t n_seq = table->size(0), M = table->size(1);
    const int *cache_len, *pinned;
    if (!c.ints(a[1], {n_seq}, &cache_len) || !c.ints(a[4], {n_pages}, &pinned)) Py_RETURN_NONE;
    at::Tensor r[3] = {c.make({n_seq, M}, at::kInt), c.make({(n_pages + 1) / 2, 3}, at::kInt), c.make({1}, at::kInt)};
    const long long need = f_pages_workspace(n_seq, n_pages);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    Workspace ws(need, stream);
    int* o[3];
    for (int i = 0; i < 3; ++i) o[i] = static_cast<int*>(r[i].data_ptr());
    const int rc = unlocked([&] {
        return f_pages_compact(static_cast<const int*>(table->data_ptr()), cache_len, n_seq, M, table->stride(0), n_pages, P,
                               pinned, o[0], M, o[1], o[2], ws.p, need, stream);
    });
    if (rc) Py_RETURN_NONE;
    return tuple_of(r);
    END_HANDLE_TH_ERRORS
}

// pages_copy(kpages, vpages, copies): True when done
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *k, *v, *copies;
    Call c;
    if (n != 3 || !(k = cuda_tensor(a[0])) || !(v = cuda_tensor(a[1])) || !(copies = cuda_tensor(a[2])) ||
        (k->dim() != 4 && k->dim() != 5) || !c.of(k, k->dim()) || !c.shares(v) || v->sizes() != k->sizes() ||
        v->stride(-1) != 1 || copies->scalar_type() != at::kInt || copies->device() != c.device || copies->dim() != 2 ||
        copies->size(1) != 3 || !copies->is_contiguous() || !small(copies->size(0)))
        Py_RETURN_NONE;
    const int l = k->dim() == 5;
    long long st[8] = {};
    for (int i = 1 - l; i < 4; ++i) st[i] = k->stride(i - 1 + l), st[4 + i] = v->stride(i - 1 + l);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.device.index());
    const int rc = unlocked([&] {
        return f_pages_copy(k->data_ptr(), v->data_ptr(), l ? k->size(0) : 1, k->size(l), k->size(l + 1), k->size(l + 2),
                            k->size(l + 3), st, static_cast<const int*>(copies->data_ptr()), copies->size(0), c.code, stream);
    });
    if (rc) Py_RETURN_NONE;
    Py_RETURN_TRUE;
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

// bind_paged(paged, paged_workspace, norm_rope, append_paged, pages_step, pages_compact, pages_copy, pages_workspace)
PyObject* bind_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[8];
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "bind_paged takes eight addresses");
        return nullptr;
    }
    for (int i = 0; i < 8; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind_paged: a null address");
            return nullptr;
        }
    f_paged = reinterpret_cast<decltype(f_paged)>(p[0]);
    f_paged_workspace = reinterpret_cast<decltype(f_paged_workspace)>(p[1]);
    f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(p[2]);
    f_append_paged = reinterpret_cast<decltype(f_append_paged)>(p[3]);
    f_pages_step = reinterpret_cast<decltype(f_pages_step)>(p[4]);
    f_pages_compact = reinterpret_cast<decltype(f_pages_compact)>(p[5]);
    f_pages_copy = reinterpret_cast<decltype(f_pages_copy)>(p[6]);
    f_pages_workspace = reinterpret_cast<decltype(f_pages_workspace)>(p[7]);
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
    {"bind_paged", fast(bind_paged), METH_FASTCALL, nullptr},
    {"paged", fast(paged), METH_FASTCALL, nullptr},
    {"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
    {"append_paged", fast(append_paged), METH_FASTCALL, nullptr},
    {"pages_step", fast(pages_step), METH_FASTCALL, nullptr},
    {"pages_compact", fast(pages_compact), METH_FASTCALL, nullptr},
    {"pages_copy", fast(pages_copy), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
