// C-ABI shim: argument validation, kernel dispatch, TMA descriptor encoding,
// decode workspace and the device status word.  The contract of every entry
// point is documented in include/attn.h.
#include "attn.h"
#include "kernels.h"
#include "paged.h"
#include "rope_turns.h"
#include "ptx.cuh"

#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <mutex>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

namespace attn {
namespace {

constexpr int kMaxDevices = 64;

thread_local char g_last_error[512] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(cudaError_t e, const char *what) {
    return fail(ATTN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte ranges [a, a + na) and [b, b + nb) overlap?
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Largest stride in elements and extent in bytes that the checks below take:
// their sums and products then stay within 64 bits.
constexpr long long kMaxStride = 1LL << 56;
constexpr double kMaxExtent = 4.0e18;

// A strided (n_outer, n_inner) set of rows of D elements: row (i, j) starts at
// element i * so + j * si.  Strides of a dimension of one entry are ignored; one
// out of range becomes -1, which rows_distinct refuses.
struct Rows {
    const char *p;
    long long n_outer, n_inner, so, si;  // strides in bytes after make_rows
    long long row;                       // bytes of one row
};

Rows make_rows(const void *p, long long n_outer, long long n_inner, long long so, long long si, long long D,
               long long esz) {
    so = so < 0 || so > kMaxStride ? -1 : so * esz;
    si = si < 0 || si > kMaxStride ? -1 : si * esz;
    Rows r{static_cast<const char *>(p), n_outer, n_inner, so, si, D * esz};
    if (n_inner == 1) r.si = r.row;
    if (n_outer == 1) r.so = r.si * n_inner > r.row ? r.si * n_inner : r.row;
    return r;
}

// No two rows share a byte: one dimension's rows fit inside the other's stride.
bool rows_distinct(const Rows &r) {
    if (r.n_outer <= 0 || r.n_inner <= 0) return true;
    if (r.so < 0 || r.si < 0 ||
        static_cast<double>(r.n_outer) * static_cast<double>(r.so) + static_cast<double>(r.n_inner) * static_cast<double>(r.si) > kMaxExtent)
        return false;
    return (r.si >= r.row && r.so >= (r.n_inner - 1) * r.si + r.row) ||
           (r.so >= r.row && r.si >= (r.n_outer - 1) * r.so + r.row);
}

// May rows of a and b share a byte?  Disjoint extents, or two runs of columns
// of one matrix (slices of a fused projection) are the cases known not to.
bool rows_overlap(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.n_outer <= 0 || b.n_outer <= 0 || a.n_inner <= 0 || b.n_inner <= 0) return false;
    auto extent = [](const Rows &r) { return (r.n_outer - 1) * r.so + (r.n_inner - 1) * r.si + r.row; };
    if (!overlaps(a.p, static_cast<size_t>(extent(a)), b.p, static_cast<size_t>(extent(b)))) return false;
    // columns [0, wa) of a and [off, off + wb) of b in rows of `period` bytes
    auto columns_apart = [](const Rows &x, const Rows &y, bool outer) {
        const long long period = outer ? x.so : x.si;
        if (period != (outer ? y.so : y.si) || period <= 0) return false;
        const long long wx = outer ? (x.n_inner - 1) * x.si + x.row : (x.n_outer - 1) * x.so + x.row;
        const long long wy = outer ? (y.n_inner - 1) * y.si + y.row : (y.n_outer - 1) * y.so + y.row;
        const long long d = static_cast<long long>(y.p - x.p);
        const long long off = ((d % period) + period) % period;
        return off >= wx && off + wy <= period;
    };
    return !columns_apart(a, b, true) && !columns_apart(a, b, false);
}

bool same_rows(const Rows &a, const Rows &b) { return a.p == b.p && a.so == b.so && a.si == b.si; }

// ------------------------------------------------------------ device status word

__device__ int g_status_word;

std::mutex g_mutex;
int *g_status_ptr[kMaxDevices];
int g_num_sms[kMaxDevices];

int current_device(int *dev) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (*dev < 0 || *dev >= kMaxDevices) return fail(ATTN_EUNSUPPORTED, "device ordinal %d out of range", *dev);
    return ATTN_OK;
}

int status_word(int **out) {
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_status_ptr[dev]) {
        void *p = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&p, g_status_word);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status word)");
        g_status_ptr[dev] = static_cast<int *>(p);
    }
    *out = g_status_ptr[dev];
    return ATTN_OK;
}

int num_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_num_sms[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        g_num_sms[dev] = n;
    }
    return g_num_sms[dev];
}

// ------------------------------------------------------------ TMA descriptors

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn g_encode = nullptr;

int get_encode(EncodeTiledFn *fn) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_encode) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                         cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !p)
            return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled entry point unavailable");
        g_encode = reinterpret_cast<EncodeTiledFn>(p);
    }
    *fn = g_encode;
    return ATTN_OK;
}

// (D, S, B*H) bf16 view of a (B, H, S, D) tensor; boxes of 64 x box_rows x 1
// with 128-byte swizzle, out-of-range rows read as zero.
int make_map(CUtensorMap *map, const void *base, int D, int S, long long BH, int box_rows = 128) {
    EncodeTiledFn encode;
    int rc = get_encode(&encode);
    if (rc) return rc;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(S),
                                static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                   static_cast<cuuint64_t>(S) * D * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return ATTN_OK;
}

// (D, rows) bf16 view of a row-major (rows, D) tensor; boxes of 64 x 128 with
// 128-byte swizzle, rows past the end read as zero.
int make_map_rows(CUtensorMap *map, const void *base, int D, long long rows) {
    EncodeTiledFn encode;
    int rc = get_encode(&encode);
    if (rc) return rc;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[2] = {64, 128};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled (2-D) failed (%d)", static_cast<int>(r));
    return ATTN_OK;
}

// (D, T, heads) bf16 view of (T, heads, D) rows with byte strides; boxes of
// 64 x 128 x 1 with 128-byte swizzle, rows past the end read as zero.
int make_map_packed(CUtensorMap *map, const Rows &r, int D) {
    EncodeTiledFn encode;
    int rc = get_encode(&encode);
    if (rc) return rc;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(r.n_outer),
                                static_cast<cuuint64_t>(r.n_inner)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(r.so), static_cast<cuuint64_t>(r.si)};
    const cuuint32_t box[3] = {64, 128, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult e = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char *>(r.p), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e != CUDA_SUCCESS) return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled (packed) failed (%d)", static_cast<int>(e));
    return ATTN_OK;
}

// (D, heads, T) bf16 view of (T, heads, D) rows with byte strides; boxes of 64 x heads x
// tokens with 128-byte swizzle: a token's heads are consecutive rows.
int make_map_tokens(CUtensorMap *map, const Rows &r, int D, int heads, int tokens) {
    EncodeTiledFn encode;
    int rc = get_encode(&encode);
    if (rc) return rc;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(r.n_inner),
                                static_cast<cuuint64_t>(r.n_outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(r.si), static_cast<cuuint64_t>(r.so)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult e = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char *>(r.p), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e != CUDA_SUCCESS) return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled (tokens) failed (%d)", static_cast<int>(e));
    return ATTN_OK;
}

// ------------------------------------------------------------ paged caches

// A pool of pages: (layers, n_pages, H_kv, P) rows of D elements, strides in bytes.
struct Pool {
    const char *p;
    long long n[4], st[4], row;
};

// strides: elements from page to page, head to head and row to row (NULL: contiguous).
// False when a stride is out of range.
bool make_pool(Pool *o, const void *p, int layers, long long layer_stride, int n_pages, int H_kv, int P, int D, long long esz,
               const long long *strides) {
    const long long dense[4] = {1LL * n_pages * H_kv * P * D, 1LL * H_kv * P * D, 1LL * P * D, D};
    const long long n[4] = {layers, n_pages, H_kv, P};
    o->p = static_cast<const char *>(p);
    o->row = D * esz;
    double extent = static_cast<double>(o->row);
    for (int i = 0; i < 4; ++i) {
        const long long s = n[i] <= 1 ? dense[i] : !strides ? dense[i] : i == 0 ? layer_stride : strides[i - 1];
        if (s < 0 || s > kMaxStride) return false;
        o->n[i] = n[i];
        o->st[i] = s * esz;
        extent += static_cast<double>(n[i]) * static_cast<double>(o->st[i]);
    }
    return extent <= kMaxExtent;
}
bool pool_empty(const Pool &o) { return o.n[0] < 1 || o.n[1] < 1 || o.n[2] < 1 || o.n[3] < 1; }
size_t pool_extent(const Pool &o) {
    if (pool_empty(o)) return 0;
    long long e = o.row;
    for (int i = 0; i < 4; ++i) e += (o.n[i] - 1) * o.st[i];
    return static_cast<size_t>(e);
}
// `dims` runs of rows nested in one another: sorted by stride, each one clears the extent of
// the smaller ones.
bool nested_distinct(long long *n, long long *st, int dims, long long row) {
    long long extent = row;
    for (int i = 0; i < dims; ++i) {
        for (int y = i + 1; y < dims; ++y)
            if (st[y] < st[i]) {
                const long long t = st[i], c = n[i];
                st[i] = st[y], n[i] = n[y], st[y] = t, n[y] = c;
            }
        if (n[i] <= 1) continue;
        if (st[i] < extent) return false;
        extent += (n[i] - 1) * st[i];
    }
    return true;
}
bool pool_distinct(const Pool &o) {
    long long n[4], st[4];
    for (int i = 0; i < 4; ++i) n[i] = o.n[i], st[i] = o.st[i];
    return pool_empty(o) || nested_distinct(n, st, 4, o.row);
}
// May rows of two pools share a byte?  Known not to: extents apart, or two halves of one
// tensor (the same strides, and the step from one to the other nested among them).
bool pools_overlap(const Pool &a, const Pool &b) {
    if (pool_empty(a) || pool_empty(b)) return false;
    if (!overlaps(a.p, pool_extent(a), b.p, pool_extent(b))) return false;
    long long n[5], st[5];
    for (int i = 0; i < 4; ++i) {
        if (a.st[i] != b.st[i] || a.n[i] != b.n[i]) return true;
        n[i] = a.n[i], st[i] = a.st[i];
    }
    n[4] = 2, st[4] = a.p < b.p ? b.p - a.p : a.p - b.p;
    return !nested_distinct(n, st, 5, a.row);
}

// The int32 arrays that say where a call's rows lie (NULL: not given, or nothing of it is read).
// Other blocks, and kernels that follow, still read them when the first rows are written.
struct Index {
    const int32_t *p;
    long long n;
    const char *name;
};
Index table_index(const int32_t *page_table, int n_pages, int n_seq, int max_pages, long long table_stride) {
    return {n_pages > 0 ? page_table : nullptr, (n_seq - 1) * (n_seq > 1 ? table_stride : 0) + max_pages, "page_table"};
}
// The name of the first that `rows` may share a byte with, or NULL.
template <int N>
const char *index_under(const Rows &rows, const Index (&index)[N]) {
    for (const Index &x : index)
        if (rows_overlap(rows, make_rows(x.p, 1, 1, x.n, x.n, x.n, 4))) return x.name;
    return nullptr;
}

// Are the heads of all pages evenly spaced?  Then head h of page p is entry p * pstep +
// h * hstep of a list of `n` heads `stride` bytes apart.
struct Heads {
    long long n, stride, pstep, hstep;
};
bool even_heads(const Pool &o, Heads *e) {
    const long long page = o.st[1], head = o.st[2];
    if (o.n[2] == 1)
        *e = {o.n[1], page, 1, 0};
    else if (o.n[1] == 1)
        *e = {o.n[2], head, 0, 1};
    else if (head > 0 && page % head == 0)
        *e = {0, head, page / head, 1};
    else if (page > 0 && head % page == 0)
        *e = {0, page, 1, head / page};
    else
        return false;
    if (e->n == 0) e->n = (o.n[1] - 1) * e->pstep + (o.n[2] - 1) * e->hstep + 1;
    return e->n <= 0x7fffffff;
}

// bf16 view of one layer of pages with 128-byte swizzle, for boxes of `rows` rows and all
// columns: (64, 8, D / 64, P / 8, heads), so that a box arrives as groups of 8 rows, in each
// the 64-column blocks.  Without even heads (e = NULL) (D, P, H_kv, n_pages) with boxes of
// one such block.  Pages out of range read as zeros.
int make_map_pages(CUtensorMap *map, const Pool &o, const Heads *e, int rows) {
    EncodeTiledFn encode;
    int rc = get_encode(&encode);
    if (rc) return rc;
    const cuuint64_t D = static_cast<cuuint64_t>(o.row / 2), P = static_cast<cuuint64_t>(o.n[3]);
    const cuuint64_t row = static_cast<cuuint64_t>(o.st[3]);
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r;
    if (e) {
        const cuuint64_t dims[5] = {64, 8, D / 64, P / 8, static_cast<cuuint64_t>(e->n)};
        const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(e->stride)};
        const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(rows / 8), 1};
        r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<char *>(o.p), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        const cuuint64_t dims[4] = {D, P, static_cast<cuuint64_t>(o.n[2]), static_cast<cuuint64_t>(o.n[1])};
        const cuuint64_t strides[3] = {row, static_cast<cuuint64_t>(o.st[2]), static_cast<cuuint64_t>(o.st[1])};
        const cuuint32_t box[4] = {64, 8, 1, 1};
        r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<char *>(o.p), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) return fail(ATTN_ECUDA, "cuTensorMapEncodeTiled (pages) failed (%d)", static_cast<int>(r));
    return ATTN_OK;
}

// ------------------------------------------------------------ decode workspace

// The decode partials.  A buffer the workspace outgrows is kept on the
// retired list, not freed: a CUDA graph captured earlier may still write to
// it on every replay.  attn_release frees them all.
constexpr int kMaxRetired = 64;
struct Workspace {
    void *ptr = nullptr;
    size_t bytes = 0;
    void *retired[kMaxRetired] = {};
    int n_retired = 0;
};
Workspace g_ws[kMaxDevices];

int workspace(size_t bytes, cudaStream_t stream, void **out) {
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mutex);
    Workspace &w = g_ws[dev];
    if (w.bytes < bytes) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(stream, &cap);
        if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
        if (cap != cudaStreamCaptureStatusNone)
            return fail(ATTN_EINVAL,
                        "attn_decode: a captured call needs %zu bytes of workspace but the device has %zu; "
                        "make one ordinary call of this size before capturing",
                        bytes, w.bytes);
        if (w.ptr && w.n_retired == kMaxRetired)
            return fail(ATTN_ENOMEM, "attn_decode: the workspace grew %d times; call attn_release", kMaxRetired);
        // grow at least geometrically, so retired buffers add up to less than the live one
        const size_t want = bytes > 2 * w.bytes ? bytes : 2 * w.bytes;
        void *p = nullptr;
        e = cudaMalloc(&p, want);
        if (e != cudaSuccess)
            return fail(ATTN_ENOMEM, "decode workspace of %zu bytes: %s", want, cudaGetErrorString(e));
        if (w.ptr) w.retired[w.n_retired++] = w.ptr;
        w.ptr = p;
        w.bytes = want;
    }
    *out = w.ptr;
    return ATTN_OK;
}

// ------------------------------------------------------------ host-buffer prefill

// Chunks per call (about) and the smallest chunk worth a copy of its own.
#ifndef ATTN_HOST_CHUNKS
#define ATTN_HOST_CHUNKS 8
#endif
constexpr int kHostChunks = ATTN_HOST_CHUNKS;
constexpr size_t kHostMinChunkBytes = 8u << 20;
constexpr int kHostEvents = 16;  // event pairs in flight; older chunks are waited for

// Per device: device copies of Q, K, V, O and kv_len (grown on demand), the
// two copy streams and the events that order them with the caller's stream.
struct HostExec {
    std::mutex mutex;
    void *buf = nullptr;
    size_t bytes = 0;
    bool ready = false;
    cudaStream_t h2d = nullptr, d2h = nullptr;
    cudaEvent_t ev[2 * kHostEvents] = {};
    cudaEvent_t ev_start = nullptr, ev_end = nullptr;

    int ensure(size_t need) {
        if (!ready) {
            cudaError_t e = cudaStreamCreateWithFlags(&h2d, cudaStreamNonBlocking);
            if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&d2h, cudaStreamNonBlocking);
            for (int i = 0; i < 2 * kHostEvents && e == cudaSuccess; ++i)
                e = cudaEventCreateWithFlags(&ev[i], cudaEventDisableTiming);
            if (e == cudaSuccess) e = cudaEventCreateWithFlags(&ev_start, cudaEventDisableTiming);
            if (e == cudaSuccess) e = cudaEventCreateWithFlags(&ev_end, cudaEventDisableTiming);
            if (e != cudaSuccess) return cuda_fail(e, "attn_fwd_host: streams and events");
            ready = true;
        }
        if (bytes < need) {
            if (buf) cudaFree(buf);  // synchronises the device: no call still uses it
            buf = nullptr;
            bytes = 0;
            cudaError_t e = cudaMalloc(&buf, need);
            if (e != cudaSuccess) {
                buf = nullptr;
                return fail(ATTN_ENOMEM, "attn_fwd_host: %zu bytes of device buffers: %s", need, cudaGetErrorString(e));
            }
            bytes = need;
        }
        return ATTN_OK;
    }
    void release() {
        std::lock_guard<std::mutex> lock(mutex);
        if (buf) cudaFree(buf);
        buf = nullptr;
        bytes = 0;
    }
};
HostExec g_host[kMaxDevices];

// Grouped-query decode: CTAs are (b, h_kv, head subgroup, chunk); the chunk
// is at most kDecodeGqaMaxChunk keys (the kernel's score buffer).
int decode_chunk_gqa(int B, int H, int H_kv, int Skv) {
    const int G = H / H_kv;
    const int gt = decode_gqa_heads_per_cta(G);
    const long long units = static_cast<long long>(B) * H_kv * ((G + gt - 1) / gt);
    const long long want = 6LL * num_sms();
    int chunk = kDecodeGqaMaxChunk;
    while (chunk > 64 && units * ((Skv + chunk - 1) / chunk) < want) chunk /= 2;
    return chunk;
}

int decode_chunk(int B, int H, int Skv) {
    // Aim for at least ~6 CTAs per SM; shorter chunks only when the batch is small.
    const long long want = 6LL * num_sms();
    int chunk = 512;
    while (chunk > 64 && static_cast<long long>(B) * H * ((Skv + chunk - 1) / chunk) < want) chunk /= 2;
    return chunk;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

ATTN_API const char *attn_last_error(void) { return g_last_error; }

ATTN_API int attn_fwd(const void *q, const void *k, const void *v, void *out, int B, int H, int Sq,
                      int Skv, int D, float scale, int causal, const int32_t *kv_len, int dtype,
                      void *stream) {
    return attn_fwd_gqa(q, k, v, out, B, H, H, Sq, Skv, D, scale, causal, kv_len, dtype, stream);
}

// Shared by attn_fwd_gqa (chunked = 0, no lse) and attn_fwd_chunked (causal,
// kv_len = cache lengths, chunked = 1, optional lse).
static int fwd_impl(const void *q, const void *k, const void *v, void *out, float *lse, int B, int H,
                    int H_kv, int Sq, int Skv, int D, float scale, int causal, const int32_t *kv_len,
                    int chunked, int dtype, void *stream) {
    g_last_error[0] = '\0';
    if (B < 1 || H < 1 || Sq < 0 || Skv < 0)
        return fail(ATTN_EINVAL, "attn_fwd: need B >= 1, H >= 1, Sq >= 0, Skv >= 0 (got %d, %d, %d, %d)", B, H, Sq, Skv);
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "attn_fwd: H_kv must divide H (got H = %d, H_kv = %d)", H, H_kv);
    if ((Sq > 0 && (!q || !out)) || (Skv > 0 && (!k || !v)))
        return fail(ATTN_EINVAL, "attn_fwd: q and out (Sq > 0), k and v (Skv > 0) must not be NULL");
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "attn_fwd: unknown dtype %d", dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "attn_fwd: D must be positive (got %d)", D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "attn_fwd: D = %d not supported (64 or 128)", D);
    if (!(scale >= 0.f) || isinf(scale)) return fail(ATTN_EINVAL, "attn_fwd: scale must be finite and >= 0");
    if (causal != 0 && causal != 1) return fail(ATTN_EINVAL, "attn_fwd: causal must be 0 or 1");
    if (causal && Sq > Skv) return fail(ATTN_EINVAL, "attn_fwd: causal needs Sq <= Skv (got %d > %d)", Sq, Skv);
    if (kv_len && !chunked && causal && Sq != Skv)
        return fail(ATTN_EINVAL, "attn_fwd: causal kv_len needs Sq == Skv (a chunk against a cache is attn_fwd_chunked)");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(ATTN_EINVAL, "attn_fwd: lse must be 4-byte aligned");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return fail(ATTN_EINVAL, "attn_fwd: q, k, v and out must be 16-byte aligned");
    if (kv_len && (reinterpret_cast<uintptr_t>(kv_len) & 3u))
        return fail(ATTN_EINVAL, "attn_fwd: kv_len must be 4-byte aligned");
    const long long bh = static_cast<long long>(B) * H;
    const long long rows = bh * (Sq > Skv ? Sq : Skv);
    if (rows >= (1LL << 31) || bh > 65535LL * 65535LL)
        return fail(ATTN_EINVAL, "attn_fwd: B*H*S = %lld rows is too large", rows);
    const size_t esz = dtype == ATTN_BF16 ? 2 : 4;
    const long long bh_kv = static_cast<long long>(B) * H_kv;
    const size_t q_bytes = static_cast<size_t>(bh) * Sq * D * esz;
    const size_t kv_bytes = static_cast<size_t>(bh_kv) * Skv * D * esz;
    if (overlaps(out, q_bytes, q, q_bytes) || overlaps(out, q_bytes, k, kv_bytes) ||
        overlaps(out, q_bytes, v, kv_bytes))
        return fail(ATTN_EINVAL, "attn_fwd: out overlaps an input");
    const size_t lse_bytes = static_cast<size_t>(bh) * Sq * sizeof(float);
    if (lse && (overlaps(lse, lse_bytes, q, q_bytes) || overlaps(lse, lse_bytes, k, kv_bytes) ||
                overlaps(lse, lse_bytes, v, kv_bytes) || overlaps(lse, lse_bytes, out, q_bytes)))
        return fail(ATTN_EINVAL, "attn_fwd: lse overlaps another tensor");
    if (Sq == 0) return ATTN_OK;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (Skv == 0) {  // no row sees a key
        cudaError_t e = launch_zero_fill(out, q_bytes, st);
        return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_fwd zero fill");
    }
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    FwdArgs a{q, k, v, out, kv_len, B, H, Sq, Skv, D, scale, causal, status, st, num_sms(), H_kv,
              chunked, lse};
    cudaError_t e;
    if (dtype == ATTN_F32) {
        if (B > 65535 || H > 65535) return fail(ATTN_EINVAL, "attn_fwd: B and H must be <= 65535 for fp32");
        e = launch_prefill_f32(a);
    } else {
        CUtensorMap tq, tk, tv;
        if ((rc = make_map(&tq, q, D, Sq, bh)) || (rc = make_map(&tk, k, D, Skv, bh_kv)) ||
            (rc = make_map(&tv, v, D, Skv, bh_kv)))
            return rc;
        e = launch_prefill_tc(a, tq, tk, tv);
    }
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_fwd launch");
}

ATTN_API int attn_fwd_gqa(const void *q, const void *k, const void *v, void *out, int B, int H,
                          int H_kv, int Sq, int Skv, int D, float scale, int causal,
                          const int32_t *kv_len, int dtype, void *stream) {
    return fwd_impl(q, k, v, out, nullptr, B, H, H_kv, Sq, Skv, D, scale, causal, kv_len, 0, dtype,
                    stream);
}

// Prefill from host buffers: the batch is cut into chunks of whole
// key/value-head groups (runs of consecutive (b, h) slices, contiguous in the
// (B, H, S, D) layout), and chunk c's copy in, chunk c - 1's attention and
// chunk c - 2's copy out run at the same time on three streams.
ATTN_API int attn_fwd_host(const void *q, const void *k, const void *v, void *out, int B, int H,
                           int H_kv, int Sq, int Skv, int D, float scale, int causal,
                           const int32_t *kv_len, int dtype, void *stream) {
    g_last_error[0] = '\0';
    if (B < 1 || H < 1 || Sq < 0 || Skv < 0)
        return fail(ATTN_EINVAL, "attn_fwd_host: need B >= 1, H >= 1, Sq >= 0, Skv >= 0");
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "attn_fwd_host: H_kv must divide H (got H = %d, H_kv = %d)", H, H_kv);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "attn_fwd_host: unknown dtype %d", dtype);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "attn_fwd_host: D = %d not supported (64 or 128)", D);
    if ((Sq > 0 && (!q || !out)) || (Skv > 0 && (!k || !v)))
        return fail(ATTN_EINVAL, "attn_fwd_host: q and out (Sq > 0), k and v (Skv > 0) must not be NULL");
    if (causal && Sq > Skv) return fail(ATTN_EINVAL, "attn_fwd_host: causal needs Sq <= Skv (got %d > %d)", Sq, Skv);
    if (kv_len && causal && Sq != Skv) return fail(ATTN_EINVAL, "attn_fwd_host: causal kv_len needs Sq == Skv");
    if (Sq == 0) return ATTN_OK;
    const size_t esz = dtype == ATTN_BF16 ? 2 : 4;
    const int G = H / H_kv;
    const size_t q_head = static_cast<size_t>(Sq) * D * esz, kv_head = static_cast<size_t>(Skv) * D * esz;
    const size_t q_bytes = static_cast<size_t>(B) * H * q_head, kv_bytes = static_cast<size_t>(B) * H_kv * kv_head;
    if (overlaps(out, q_bytes, q, q_bytes) || overlaps(out, q_bytes, k, kv_bytes) || overlaps(out, q_bytes, v, kv_bytes))
        return fail(ATTN_EINVAL, "attn_fwd_host: out overlaps an input");
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    HostExec &x = g_host[dev];
    std::lock_guard<std::mutex> lock(x.mutex);  // one call at a time per device: it owns the buffers
    // device copies: Q | K | V | O | kv_len, each 256-byte aligned
    auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    const size_t off_k = up(q_bytes), off_v = off_k + up(kv_bytes), off_o = off_v + up(kv_bytes);
    const size_t off_l = off_o + up(q_bytes), total = off_l + up(static_cast<size_t>(B) * sizeof(int32_t));
    if ((rc = x.ensure(total))) return rc;
    char *dbuf = static_cast<char *>(x.buf);
    int32_t *d_len = kv_len ? reinterpret_cast<int32_t *>(dbuf + off_l) : nullptr;
    // chunks: whole batches when one batch is below the target, else runs of key/value heads of one batch
    const size_t per_b = static_cast<size_t>(H) * q_head + 2 * static_cast<size_t>(H_kv) * kv_head;
    size_t target = (static_cast<size_t>(B) * per_b) / kHostChunks;
    target = target < kHostMinChunkBytes ? kHostMinChunkBytes : target;
    int nb = 1, kv_per = H_kv;  // batches per chunk, or key/value heads per chunk (nb == 1)
    if (per_b <= target) {
        nb = static_cast<int>(target / per_b);
        nb = nb < 1 ? 1 : (nb > B ? B : nb);
    } else {
        const size_t per_kv = static_cast<size_t>(G) * q_head + 2 * kv_head;
        kv_per = static_cast<int>((target + per_kv - 1) / per_kv);
        kv_per = kv_per < 1 ? 1 : (kv_per > H_kv ? H_kv : kv_per);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaEventRecord(x.ev_start, st);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(x.h2d, x.ev_start, 0);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(x.d2h, x.ev_start, 0);
    if (e == cudaSuccess && kv_len)
        e = cudaMemcpyAsync(d_len, kv_len, static_cast<size_t>(B) * sizeof(int32_t), cudaMemcpyHostToDevice, x.h2d);
    int n_chunk = 0;
    for (int b0 = 0; b0 < B && e == cudaSuccess && rc == ATTN_OK; b0 += nb) {
        const int bn = b0 + nb <= B ? nb : B - b0;
        for (int g0 = 0; g0 < H_kv && e == cudaSuccess && rc == ATTN_OK; g0 += kv_per) {
            const int gn = g0 + kv_per <= H_kv ? kv_per : H_kv - g0;
            // slices: batches [b0, b0 + bn) x kv heads [g0, g0 + gn) (nb == 1 or gn == H_kv)
            const size_t qo = (static_cast<size_t>(b0) * H + static_cast<size_t>(g0) * G) * q_head;
            const size_t ko = (static_cast<size_t>(b0) * H_kv + g0) * kv_head;
            const size_t qn = static_cast<size_t>(bn) * gn * G * q_head, kn = static_cast<size_t>(bn) * gn * kv_head;
            cudaEvent_t ev_in = x.ev[2 * (n_chunk % kHostEvents)], ev_done = x.ev[2 * (n_chunk % kHostEvents) + 1];
            if (n_chunk >= kHostEvents) e = cudaEventSynchronize(x.ev[2 * (n_chunk % kHostEvents) + 1]);
            if (e == cudaSuccess) e = cudaMemcpyAsync(dbuf + qo, static_cast<const char *>(q) + qo, qn, cudaMemcpyHostToDevice, x.h2d);
            if (e == cudaSuccess && Skv > 0)
                e = cudaMemcpyAsync(dbuf + off_k + ko, static_cast<const char *>(k) + ko, kn, cudaMemcpyHostToDevice, x.h2d);
            if (e == cudaSuccess && Skv > 0)
                e = cudaMemcpyAsync(dbuf + off_v + ko, static_cast<const char *>(v) + ko, kn, cudaMemcpyHostToDevice, x.h2d);
            if (e == cudaSuccess) e = cudaEventRecord(ev_in, x.h2d);
            if (e == cudaSuccess) e = cudaStreamWaitEvent(st, ev_in, 0);
            if (e != cudaSuccess) break;
            rc = fwd_impl(dbuf + qo, dbuf + off_k + ko, dbuf + off_v + ko, dbuf + off_o + qo, nullptr, bn,
                          gn * G, gn, Sq, Skv, D, scale, causal, d_len ? d_len + b0 : nullptr, 0, dtype, st);
            if (rc) break;
            e = cudaEventRecord(ev_done, st);
            if (e == cudaSuccess) e = cudaStreamWaitEvent(x.d2h, ev_done, 0);
            if (e == cudaSuccess)
                e = cudaMemcpyAsync(static_cast<char *>(out) + qo, dbuf + off_o + qo, qn, cudaMemcpyDeviceToHost, x.d2h);
            ++n_chunk;
        }
    }
    // the caller's stream resumes after the last copy out; the call returns when it is done
    cudaError_t e2 = cudaEventRecord(x.ev_end, x.d2h);
    if (e2 == cudaSuccess) e2 = cudaStreamWaitEvent(st, x.ev_end, 0);
    if (e2 == cudaSuccess) e2 = cudaEventSynchronize(x.ev_end);
    if (rc) return rc;
    if (e != cudaSuccess) return cuda_fail(e, "attn_fwd_host");
    if (e2 != cudaSuccess) return cuda_fail(e2, "attn_fwd_host (completion)");
    return ATTN_OK;
}

ATTN_API int attn_fwd_chunked(const void *q, const void *kcache, const void *vcache, void *out,
                              float *lse, int B, int H, int H_kv, int Sq, int Skv, int D, float scale,
                              const int32_t *cache_len, int dtype, void *stream) {
    return fwd_impl(q, kcache, vcache, out, lse, B, H, H_kv, Sq, Skv, D, scale, 1, cache_len, 1, dtype,
                    stream);
}

ATTN_API int attn_fwd_debug(const void *q, const void *k, const void *v, void *out, float *weights,
                            int B, int H, int H_kv, int Sq, int Skv, int Dk, int Dv, float scale,
                            int causal, const int32_t *kv_len, int dtype, void *stream) {
    g_last_error[0] = '\0';
    if (B < 1 || H < 1 || Sq < 0 || Skv < 0)
        return fail(ATTN_EINVAL, "attn_fwd_debug: need B >= 1, H >= 1, Sq >= 0, Skv >= 0");
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "attn_fwd_debug: H_kv must divide H (got H = %d, H_kv = %d)", H, H_kv);
    if (Dk < 1 || Dk > 256 || Dv < 1 || Dv > 256)
        return fail(ATTN_EINVAL, "attn_fwd_debug: Dk and Dv must be in [1, 256] (got %d, %d)", Dk, Dv);
    if (Skv > 16384) return fail(ATTN_EUNSUPPORTED, "attn_fwd_debug: Skv = %d above 16384", Skv);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "attn_fwd_debug: unknown dtype %d", dtype);
    if (!(scale >= 0.f) || isinf(scale)) return fail(ATTN_EINVAL, "attn_fwd_debug: scale must be finite and >= 0");
    if (causal != 0 && causal != 1) return fail(ATTN_EINVAL, "attn_fwd_debug: causal must be 0 or 1");
    if (causal && Sq > Skv) return fail(ATTN_EINVAL, "attn_fwd_debug: causal needs Sq <= Skv (got %d > %d)", Sq, Skv);
    if (kv_len && causal && Sq != Skv)
        return fail(ATTN_EINVAL, "attn_fwd_debug: causal kv_len needs Sq == Skv");
    if ((Sq > 0 && (!q || !out)) || (Skv > 0 && (!k || !v)))
        return fail(ATTN_EINVAL, "attn_fwd_debug: q and out (Sq > 0), k and v (Skv > 0) must not be NULL");
    const size_t esz = dtype == ATTN_BF16 ? 2 : 4;
    const uintptr_t amask = esz - 1;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(out)) & amask)
        return fail(ATTN_EINVAL, "attn_fwd_debug: tensors must be aligned to their element size");
    if ((kv_len && (reinterpret_cast<uintptr_t>(kv_len) & 3u)) || (weights && (reinterpret_cast<uintptr_t>(weights) & 3u)))
        return fail(ATTN_EINVAL, "attn_fwd_debug: kv_len and weights must be 4-byte aligned");
    const long long rows = static_cast<long long>(B) * H * Sq;
    if (rows >= (1LL << 31)) return fail(ATTN_EINVAL, "attn_fwd_debug: B*H*Sq is too large");
    const long long bh_kv = static_cast<long long>(B) * H_kv;
    const size_t q_bytes = static_cast<size_t>(rows) * Dk * esz, o_bytes = static_cast<size_t>(rows) * Dv * esz;
    const size_t k_bytes = static_cast<size_t>(bh_kv) * Skv * Dk * esz, v_bytes = static_cast<size_t>(bh_kv) * Skv * Dv * esz;
    const size_t w_bytes = static_cast<size_t>(rows) * Skv * sizeof(float);
    if (overlaps(out, o_bytes, q, q_bytes) || overlaps(out, o_bytes, k, k_bytes) || overlaps(out, o_bytes, v, v_bytes) ||
        (weights && (overlaps(weights, w_bytes, q, q_bytes) || overlaps(weights, w_bytes, k, k_bytes) ||
                     overlaps(weights, w_bytes, v, v_bytes) || overlaps(weights, w_bytes, out, o_bytes))))
        return fail(ATTN_EINVAL, "attn_fwd_debug: out or weights overlaps another tensor");
    if (rows == 0) return ATTN_OK;
    DebugArgs a{q, k, v, out, weights, kv_len, B, H, H_kv, Sq, Skv, Dk, Dv, scale, causal,
                dtype == ATTN_BF16 ? 1 : 0, static_cast<cudaStream_t>(stream)};
    const cudaError_t e = launch_debug_attention(a);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_fwd_debug launch");
}

ATTN_API int attn_decode_splits(int B, int H, int Skv, int D) {
    if (B < 1 || H < 1 || Skv < 0 || (D != 64 && D != 128)) return ATTN_EINVAL;
    const int chunk = decode_chunk(B, H, Skv);
    const int n = (Skv + chunk - 1) / chunk;
    return n > 0 ? n : 1;
}

ATTN_API int attn_decode(const void *q, const void *kcache, const void *vcache, void *out, int B,
                         int H, int Skv, int D, const int32_t *kv_len, int dtype, void *stream) {
    return attn_decode_gqa(q, kcache, vcache, out, B, H, H, Skv, D, kv_len, dtype, stream);
}

ATTN_API int attn_decode_gqa(const void *q, const void *kcache, const void *vcache, void *out, int B,
                             int H, int H_kv, int Skv, int D, const int32_t *kv_len, int dtype,
                             void *stream) {
    g_last_error[0] = '\0';
    if (B < 1 || H < 1 || Skv < 0)
        return fail(ATTN_EINVAL, "attn_decode: need B >= 1, H >= 1, Skv >= 0 (got %d, %d, %d)", B, H, Skv);
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "attn_decode: H_kv must divide H (got H = %d, H_kv = %d)", H, H_kv);
    if (!q || !out || (Skv > 0 && (!kcache || !vcache)))
        return fail(ATTN_EINVAL, "attn_decode: q, out and (for Skv > 0) kcache, vcache must not be NULL");
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "attn_decode: unknown dtype %d", dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "attn_decode: D must be positive (got %d)", D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "attn_decode: D = %d not supported (64 or 128)", D);
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(out))
        return fail(ATTN_EINVAL, "attn_decode: q, kcache, vcache and out must be 16-byte aligned");
    if (kv_len && (reinterpret_cast<uintptr_t>(kv_len) & 3u))
        return fail(ATTN_EINVAL, "attn_decode: kv_len must be 4-byte aligned");
    const long long bh = static_cast<long long>(B) * H;
    const long long bh_kv = static_cast<long long>(B) * H_kv;
    if (bh * (Skv > 1 ? Skv : 1) >= (1LL << 31) || bh >= (1LL << 31) / 64)
        return fail(ATTN_EINVAL, "attn_decode: B*H*Skv is too large");
    const size_t esz = dtype == ATTN_BF16 ? 2 : 4;
    const size_t qo_bytes = static_cast<size_t>(bh) * D * esz;
    const size_t kv_bytes = static_cast<size_t>(bh_kv) * Skv * D * esz;
    if (overlaps(out, qo_bytes, q, qo_bytes) || overlaps(out, qo_bytes, kcache, kv_bytes) ||
        overlaps(out, qo_bytes, vcache, kv_bytes))
        return fail(ATTN_EINVAL, "attn_decode: out overlaps an input");

    // bf16 with large query groups: the tensor-core kernel (the group's queries
    // are the rows of one tile); fp32: its own CUDA-core kernel
    const bool f32 = dtype == ATTN_F32;
    const int G = H / H_kv;
    const bool tc = !f32 && G >= kDecodeTcMinGroup && G <= 128 && bh_kv <= 65535;
    const int chunk = tc ? decode_tc_chunk(B, H_kv, Skv, num_sms())
                         : ((H_kv == H || f32) ? decode_chunk(B, H, Skv) : decode_chunk_gqa(B, H, H_kv, Skv));
    const int n_split = Skv > 0 ? (Skv + chunk - 1) / chunk : 1;
    const size_t o_bytes = static_cast<size_t>(bh) * n_split * D * sizeof(float);
    const size_t ml_bytes = static_cast<size_t>(bh) * n_split * 2 * sizeof(float);
    void *ws = nullptr;
    int rc = workspace(o_bytes + ml_bytes, static_cast<cudaStream_t>(stream), &ws);
    if (rc) return rc;
    int *status = nullptr;
    if ((rc = status_word(&status))) return rc;
    DecodeArgs a{q, kcache, vcache, out, kv_len, B, H, Skv, D, 1.0f / sqrtf(static_cast<float>(D)),
                 chunk, n_split, static_cast<float *>(ws),
                 reinterpret_cast<float *>(static_cast<char *>(ws) + o_bytes), status,
                 static_cast<cudaStream_t>(stream), H_kv};
    cudaError_t e;
    if (tc) {
        CUtensorMap tq, tk, tv;
        if (Skv > 0 && ((rc = make_map_rows(&tq, q, D, bh)) || (rc = make_map(&tk, kcache, D, Skv, bh_kv, 64)) ||
                        (rc = make_map(&tv, vcache, D, Skv, bh_kv, 64))))
            return rc;
        e = launch_decode_tc(a, tq, tk, tv);
    } else if (f32) {
        e = launch_decode_f32(a);
    } else {
        e = H_kv == H ? launch_decode(a) : launch_decode_gqa(a);
    }
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_decode launch");
}

ATTN_API int attn_decode_noalloc(const void *q, const void *kcache, const void *vcache, void *out, int B,
                                 int H, int Skv, int D, const int32_t *kv_len, int dtype, void *stream) {
    g_last_error[0] = '\0';
    if (B < 1 || H < 1 || Skv < 0)
        return fail(ATTN_EINVAL, "attn_decode_noalloc: need B >= 1, H >= 1, Skv >= 0 (got %d, %d, %d)", B, H, Skv);
    if (!q || !out || (Skv > 0 && (!kcache || !vcache)))
        return fail(ATTN_EINVAL, "attn_decode_noalloc: q, out and (for Skv > 0) kcache, vcache must not be NULL");
    if (dtype != ATTN_F32 && dtype != ATTN_BF16)
        return fail(ATTN_EINVAL, "attn_decode_noalloc: unknown dtype %d", dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "attn_decode_noalloc: D must be positive (got %d)", D);
    if (D != 64 && D != 128)
        return fail(ATTN_EUNSUPPORTED, "attn_decode_noalloc: D = %d not supported (64 or 128)", D);
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(out))
        return fail(ATTN_EINVAL, "attn_decode_noalloc: q, kcache, vcache and out must be 16-byte aligned");
    if (kv_len && (reinterpret_cast<uintptr_t>(kv_len) & 3u))
        return fail(ATTN_EINVAL, "attn_decode_noalloc: kv_len must be 4-byte aligned");
    const long long bh = static_cast<long long>(B) * H;
    if (bh * (Skv > 1 ? Skv : 1) >= (1LL << 31) || bh >= (1LL << 31) / 64)
        return fail(ATTN_EINVAL, "attn_decode_noalloc: B*H*Skv is too large");
    const size_t esz = dtype == ATTN_BF16 ? 2 : 4;
    const size_t qo_bytes = static_cast<size_t>(bh) * D * esz;
    const size_t kv_bytes = static_cast<size_t>(bh) * Skv * D * esz;
    if (overlaps(out, qo_bytes, q, qo_bytes) || overlaps(out, qo_bytes, kcache, kv_bytes) ||
        overlaps(out, qo_bytes, vcache, kv_bytes))
        return fail(ATTN_EINVAL, "attn_decode_noalloc: out overlaps an input");
    const int chunk = decode_chunk(B, H, Skv);
    const int n_split = attn_decode_splits(B, H, Skv, D);
    const size_t need = static_cast<size_t>(bh) * n_split * (D + 2) * sizeof(float);
    if (need > kDecodeNoAllocScratchBytes)
        return fail(ATTN_EINVAL,
                    "attn_decode_noalloc: these sizes need %zu bytes of scratch; the library's fixed "
                    "scratch holds %zu (use attn_decode, or fewer sequences per call)",
                    need, kDecodeNoAllocScratchBytes);
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    DecodeArgs a{q, kcache, vcache, out, kv_len, B, H, Skv, D, 1.0f / sqrtf(static_cast<float>(D)),
                 chunk, n_split, nullptr, nullptr, status, static_cast<cudaStream_t>(stream), H};
    cudaError_t e = launch_decode_noalloc(a, dtype == ATTN_F32);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_decode_noalloc launch");
}

ATTN_API long long attn_fwd_packed_workspace(int T, int n_seq, int H, int H_kv, int dtype) {
    if (T < 0 || n_seq < 0 || H < 1 || H_kv < 1 || H % H_kv || (dtype != ATTN_F32 && dtype != ATTN_BF16)) return ATTN_EINVAL;
    if (dtype == ATTN_F32) return 0;
    return 16 * (1 + packed_plan_tiles(T, n_seq, packed_unit_rows(H, H_kv)));
}

ATTN_API int attn_fwd_packed(const void *q, const void *k, const void *v, void *out, float *lse, int T, int H, int H_kv,
                             int D, const long long *strides, const int32_t *cu_seqlens, int n_seq, float scale,
                             int causal, int dtype, void *workspace, long long workspace_bytes, void *stream) {
    g_last_error[0] = '\0';
    const char *who = "attn_fwd_packed";
    if (T < 0 || n_seq < 0 || H < 1) return fail(ATTN_EINVAL, "%s: need T >= 0, n_seq >= 0, H >= 1", who);
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "%s: H_kv must divide H (got H = %d, H_kv = %d)", who, H, H_kv);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, D);
    if (!(scale >= 0.f) || isinf(scale)) return fail(ATTN_EINVAL, "%s: scale must be finite and >= 0", who);
    if (causal != 0 && causal != 1) return fail(ATTN_EINVAL, "%s: causal must be 0 or 1", who);
    if (T == 0 || n_seq == 0) return ATTN_OK;
    if (!q || !k || !v || !out || !cu_seqlens) return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return fail(ATTN_EINVAL, "%s: q, k, v and out must be 16-byte aligned", who);
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(lse)) & 3u)
        return fail(ATTN_EINVAL, "%s: cu_seqlens and lse must be 4-byte aligned", who);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    const void *ptrs[4] = {q, k, v, out};
    const int heads[4] = {H, H_kv, H_kv, H};
    const char *names[4] = {"q", "k", "v", "out"};
    Rows rows[4];
    for (int i = 0; i < 4; ++i) {
        const long long ts = strides ? strides[2 * i] : static_cast<long long>(heads[i]) * D;
        const long long hs = strides ? strides[2 * i + 1] : D;
        rows[i] = make_rows(ptrs[i], T, heads[i], ts, hs, D, esz);
        if (!rows_distinct(rows[i]) || rows[i].so >= (1LL << 40) || rows[i].si >= (1LL << 40))
            return fail(ATTN_EINVAL, "%s: the rows of %s overlap or lie too far apart (strides %lld, %lld)", who, names[i],
                        ts, hs);
        if (rows[i].so % 16 || rows[i].si % 16)
            return fail(ATTN_EINVAL, "%s: the strides of %s must be multiples of 16 bytes", who, names[i]);
    }
    for (int i = 0; i < 3; ++i)
        if (rows_overlap(rows[3], rows[i])) return fail(ATTN_EINVAL, "%s: out overlaps %s", who, names[i]);
    if (lse) {
        const Rows lr = make_rows(lse, T, 1, H, H, H, 4);
        for (int i = 0; i < 4; ++i)
            if (rows_overlap(lr, rows[i])) return fail(ATTN_EINVAL, "%s: lse overlaps %s", who, names[i]);
    }
    const long long need = attn_fwd_packed_workspace(T, n_seq, H, H_kv, dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned16(workspace))
            return fail(ATTN_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes (got %lld)", who, need,
                        workspace ? workspace_bytes : 0LL);
        const Rows wr = make_rows(workspace, 1, 1, need, need, need, 1);
        for (int i = 0; i < 4; ++i)
            if (rows_overlap(wr, rows[i])) return fail(ATTN_EINVAL, "%s: workspace overlaps %s", who, names[i]);
        if (overlaps(workspace, static_cast<size_t>(need), cu_seqlens, (static_cast<size_t>(n_seq) + 1) * 4) ||
            (lse && overlaps(workspace, static_cast<size_t>(need), lse, static_cast<size_t>(T) * H * 4)))
            return fail(ATTN_EINVAL, "%s: workspace overlaps cu_seqlens or lse", who);
    }
    const int unit = packed_unit_rows(H, H_kv);
    const long long tiles = packed_plan_tiles(T, n_seq, unit);
    if ((dtype == ATTN_F32 ? packed_f32_blocks(T, n_seq) * H : tiles * (unit == 128 ? H / 2 : H)) > 0x7fffffffLL)
        return fail(ATTN_EINVAL, "%s: %d tokens in %d sequences of %d heads are too many", who, T, n_seq, H);
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    PackedArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse;
    a.B = n_seq, a.H = H, a.H_kv = H_kv, a.Sq = T, a.Skv = T, a.D = D;
    a.scale = scale, a.causal = causal, a.status = status;
    a.stream = static_cast<cudaStream_t>(stream), a.n_sm = num_sms();
    a.cu_seqlens = cu_seqlens, a.plan = static_cast<const int4 *>(workspace);
    a.q_ts = rows[0].so / esz, a.q_hs = rows[0].si / esz, a.k_ts = rows[1].so / esz, a.k_hs = rows[1].si / esz;
    a.v_ts = rows[2].so / esz, a.v_hs = rows[2].si / esz, a.o_ts = rows[3].so / esz, a.o_hs = rows[3].si / esz;
    cudaError_t e;
    if (dtype == ATTN_F32) {
        e = launch_packed_f32(a);
    } else {
        CUtensorMap tq, tk, tv;
        if ((rc = make_map_packed(&tq, rows[0], D)) || (rc = make_map_packed(&tk, rows[1], D)) ||
            (rc = make_map_packed(&tv, rows[2], D)))
            return rc;
        e = launch_packed_tc(a, tiles, tq, tk, tv);
    }
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_fwd_packed launch");
}

// Most cache rows of a sequence: the kernels count keys in 32 bits to the end of a
// 128-key tile (bf16), or of the last of eight splits, half of them past the end (fp32).
static int tree_max_rows(int dtype) { return dtype == ATTN_BF16 ? 0x7fffff00 : 0x40000000; }

ATTN_API long long attn_decode_tree_workspace(int B, int H, int H_kv, int T, int Skv, int D, int dtype) {
    if (B < 1 || H < 1 || H_kv < 1 || H % H_kv || T < 0 || T > kTreeMaxTokens || Skv < 0 || (D != 64 && D != 128) ||
        (dtype != ATTN_F32 && dtype != ATTN_BF16))
        return ATTN_EINVAL;
    if (Skv > tree_max_rows(dtype)) return ATTN_EINVAL;
    if (T == 0 || Skv == 0) return 0;
    if (dtype == ATTN_F32) {
        const int chunk = tree_chunk_f32(B, H, H_kv, T, Skv, D, num_sms());
        const long long n_split = tree_splits_f32(Skv, chunk);
        return n_split <= kTreeClusterF32 ? 0 : static_cast<long long>(B) * H * T * n_split * (D + 2) * 4;
    }
    const long long grid = tree_tc_grid(B, H, H_kv, T, Skv, num_sms());
    if (grid < 0) return ATTN_EINVAL;
    return grid * 32 + 2 * grid * tree_tc_slot_rows(H, H_kv, T) * (D + 2) * 4;
}

ATTN_API int attn_decode_tree(const void *q, const void *kcache, const void *vcache, void *out, int B, int H, int H_kv,
                              int T, int Skv, int D, const long long *strides, const int32_t *parents,
                              int parents_stride, const int32_t *cache_len, const int32_t *draft_len, float scale,
                              int dtype, void *workspace, long long workspace_bytes, void *stream) {
    g_last_error[0] = '\0';
    const char *who = "attn_decode_tree";
    if (B < 1 || H < 1 || T < 0 || Skv < 0)
        return fail(ATTN_EINVAL, "%s: need B >= 1, H >= 1, T >= 0, Skv >= 0", who);
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "%s: H_kv must divide H (got H = %d, H_kv = %d)", who, H, H_kv);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, D);
    if (T > kTreeMaxTokens)
        return fail(ATTN_EUNSUPPORTED, "%s: T = %d drafted tokens, at most %d", who, T, kTreeMaxTokens);
    if (!(scale >= 0.f) || isinf(scale)) return fail(ATTN_EINVAL, "%s: scale must be finite and >= 0", who);
    if (parents_stride != 0 && parents_stride < T)
        return fail(ATTN_EINVAL, "%s: parents_stride must be 0 (one tree for all) or >= T", who);
    if (T == 0) return ATTN_OK;
    if (!q || !out || !parents || (Skv > 0 && (!kcache || !vcache))) return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(out))
        return fail(ATTN_EINVAL, "%s: q, kcache, vcache and out must be 16-byte aligned", who);
    if ((reinterpret_cast<uintptr_t>(parents) | reinterpret_cast<uintptr_t>(cache_len) |
         reinterpret_cast<uintptr_t>(draft_len)) & 3u)
        return fail(ATTN_EINVAL, "%s: parents, cache_len and draft_len must be 4-byte aligned", who);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    // q and out: (B, H, T) rows with three strides each
    long long st[2][3];
    for (int i = 0; i < 2; ++i) {
        st[i][0] = B == 1 ? 0 : strides ? strides[3 * i] : static_cast<long long>(H) * T * D;
        st[i][1] = H == 1 ? 0 : strides ? strides[3 * i + 1] : static_cast<long long>(T) * D;
        st[i][2] = T == 1 ? 0 : strides ? strides[3 * i + 2] : D;
        double extent = 0;
        const int count[3] = {B, H, T};
        for (int x = 0; x < 3; ++x) {
            if (st[i][x] < 0 || st[i][x] > kMaxStride)
                return fail(ATTN_EINVAL, "%s: stride %lld is negative or too large", who, st[i][x]);
            extent += static_cast<double>(count[x]) * static_cast<double>(st[i][x]) * static_cast<double>(esz);
        }
        if (extent > kMaxExtent) return fail(ATTN_EINVAL, "%s: the strides are too large", who);
        if (st[i][0] * esz % 16 || st[i][1] * esz % 16 || st[i][2] * esz % 16)
            return fail(ATTN_EINVAL, "%s: strides must be multiples of 16 bytes", who);
    }
    // rows of out must be distinct: sorted by stride, each one clears the extent of the smaller ones
    {
        long long s[3] = {st[1][0], st[1][1], st[1][2]}, n[3] = {B, H, T}, extent = D;
        for (int x = 0; x < 3; ++x)
            for (int y = x + 1; y < 3; ++y)
                if (s[y] < s[x]) {
                    const long long a = s[x], c = n[x];
                    s[x] = s[y], n[x] = n[y], s[y] = a, n[y] = c;
                }
        for (int x = 0; x < 3; ++x) {
            if (n[x] == 1) continue;
            if (s[x] < extent) return fail(ATTN_EINVAL, "%s: the rows of out overlap", who);
            extent += (n[x] - 1) * s[x];
        }
    }
    const size_t q_bytes = static_cast<size_t>(((B - 1) * st[0][0] + (H - 1) * st[0][1] + (T - 1) * st[0][2] + D) * esz);
    const size_t o_bytes = static_cast<size_t>(((B - 1) * st[1][0] + (H - 1) * st[1][1] + (T - 1) * st[1][2] + D) * esz);
    const long long bh_kv = static_cast<long long>(B) * H_kv;
    const size_t kv_bytes = static_cast<size_t>(bh_kv) * Skv * D * esz;
    if (overlaps(out, o_bytes, q, q_bytes) || overlaps(out, o_bytes, kcache, kv_bytes) ||
        overlaps(out, o_bytes, vcache, kv_bytes))
        return fail(ATTN_EINVAL, "%s: out overlaps an input", who);
    const bool f32 = dtype == ATTN_F32;
    const long long rows = static_cast<long long>(B) * H * T;
    if (rows >= (1LL << 31) || bh_kv * Skv >= (1LL << 31) || Skv > tree_max_rows(dtype)) return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    const int chunk = f32 && Skv > 0 ? tree_chunk_f32(B, H, H_kv, T, Skv, D, num_sms()) : 64;
    const int n_split = !f32 ? tree_tc_grid(B, H, H_kv, T, Skv, num_sms()) : Skv > 0 ? tree_splits_f32(Skv, chunk) : 1;
    if (n_split < 0) return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    if (f32 && bh_kv * n_split * (((H / H_kv) * static_cast<long long>(T) + 31) / 32) >= (1LL << 31))
        return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    const long long need = attn_decode_tree_workspace(B, H, H_kv, T, Skv, D, dtype);
    // rows of partial results
    const long long parts = f32 ? rows * n_split : 2LL * n_split * tree_tc_slot_rows(H, H_kv, T);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned16(workspace))
            return fail(ATTN_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes (got %lld)", who, need,
                        workspace ? workspace_bytes : 0LL);
        const size_t nb = static_cast<size_t>(need);
        if (overlaps(workspace, nb, q, q_bytes) || overlaps(workspace, nb, out, o_bytes) ||
            overlaps(workspace, nb, kcache, kv_bytes) || overlaps(workspace, nb, vcache, kv_bytes))
            return fail(ATTN_EINVAL, "%s: workspace overlaps a tensor", who);
    }
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    TreeArgs a{};
    a.q = q, a.k = kcache, a.v = vcache, a.out = out;
    a.parents = parents, a.cache_len = cache_len, a.draft_len = draft_len, a.parents_bs = parents_stride;
    a.q_bs = st[0][0], a.q_hs = st[0][1], a.q_ts = st[0][2], a.o_bs = st[1][0], a.o_hs = st[1][1], a.o_ts = st[1][2];
    a.B = B, a.H = H, a.H_kv = H_kv, a.T = T, a.Skv = Skv, a.D = D, a.scale = scale;
    a.chunk = chunk, a.n_split = n_split;
    if (need > 0) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = a.part_o + parts * D;
        a.merge = reinterpret_cast<int *>(a.part_ml + parts * 2);
    }
    a.status = status, a.stream = static_cast<cudaStream_t>(stream), a.n_sm = num_sms();
    cudaError_t e;
    if (f32) {
        e = launch_tree_f32(a);
    } else {
        CUtensorMap tk, tv;
        if (Skv > 0 && ((rc = make_map(&tk, kcache, D, Skv, bh_kv)) || (rc = make_map(&tv, vcache, D, Skv, bh_kv))))
            return rc;
        e = Skv > 0 ? launch_tree_tc(a, tk, tv) : launch_tree_zero(a);
    }
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_decode_tree launch");
}

// What the sizes of a paged call decide: rows of a tile, CTAs, splits.  n_seq, T, H, H_kv,
// D, P, max_len and `ragged` (sequences of different numbers of tokens) are given.
// Returns the bytes of workspace, or a negative code with its reason.
static long long paged_sizes(const char *who, PagedArgs &a, bool ragged, int dtype) {
    const int G = a.H / a.H_kv;
    // key / P as the upper half of key * ceil(2^32 / P): right while key times what was rounded up
    // stays below 2^32
    const unsigned long long magic = ((1ULL << 32) + a.P - 1) / a.P, over = magic * a.P - (1ULL << 32);
    a.page_magic = over * static_cast<unsigned long long>(a.max_len) < (1ULL << 32) ? static_cast<unsigned>(magic) : 0u;
    a.n_sm = num_sms();
    a.per_seq = ragged || a.n_seq < 1 ? 0 : a.T / a.n_seq;
    const long long rows = static_cast<long long>(a.T) * a.H;
    // keys are counted in 32 bits some tiles past the last one (bf16), or to the end of the last split
    if (rows >= (1LL << 31) || a.max_len > (dtype == ATTN_BF16 ? 0x7fff0000 : 0x40000000))
        return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    if (a.T == 0 || a.n_seq == 0) return 0;
    if (dtype == ATTN_F32) {
        static const int32_t some = 0;
        PagedArgs b = a;
        b.cu_seqlens = ragged ? &some : nullptr;
        const long long blocks = paged_f32_blocks(b) * a.H_kv;
        a.n_split = paged_f32_splits(b);
        if (blocks * a.n_split >= (1LL << 31) || blocks * 4 >= (1LL << 31))
            return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
        return a.n_split <= kTreeClusterF32 ? 0 : blocks * 32 * a.n_split * (a.D + 2) * 4;
    }
    a.groups = (G + 127) / 128;
    a.heads = (G + a.groups - 1) / a.groups;
    a.tokens = 128 / a.heads;
    const int most = ragged ? a.T : a.per_seq;  // tokens of a sequence
    a.box_tokens = most < a.tokens ? most : a.tokens;
    a.single = most <= a.tokens;
    a.slot_rows = a.single ? (a.box_tokens * a.heads + 31) / 32 * 32 : 256;
    a.box = 128;
    while (a.P % a.box) a.box /= 2;
    // Few units: each a cluster of eight, four, two or one CTAs, as many as the SMs hold (of
    // four and eight not on all of them: 16 of eight take 17.6 us, as one waits, 15 take 9.9).
    // Against the equal shares of all SMs, with H 32 / 8 and D 128: one sequence of 1000 keys
    // 8.6 against 13.4 us, two 9.6 and 14.2, four 11.6 and 14.9, 9 12.4 and 20.0, 16 15.0 and
    // 23.3.  Long ones lose: 42.9 and 36.0 for one of 32000, 24.3 and 20.7 for two of 8000, 24.7 and
    // 19.5 for four of 4000.  So up to 6 tiles more for the longest sequence than an equal share is,
    // where that fills its row of the table and the others are half as long.  The lengths themselves
    // are on the device: short sequences in a wide table take the equal shares (one of 1501
    // keys 9.1 us where the table has up to some 10600 tokens, 13.7 in a wider one).
    const long long units = static_cast<long long>(a.n_seq) * a.H_kv * a.groups;
    a.cluster = 0;
    for (int c = a.single ? kPagedCluster : 0; c > 0 && a.cluster == 0; c /= 2)
        if (3 * units * c <= (c < 4 ? 3LL : 2LL) * a.n_sm) a.cluster = c;
    if (a.cluster) {
        const double shared = units * (a.n_seq + 1.0) / (2.0 * a.n_seq) / a.n_sm;  // of a tile of every unit, an SM's
        if (a.max_len / 128.0 * (1.0 / a.cluster - shared) > 6.0) a.cluster = 0;
    }
    if (a.cluster) {
        a.grid = static_cast<int>(units) * a.cluster;
        a.cluster_shift = a.cluster == 8 ? 3 : a.cluster == 4 ? 2 : a.cluster == 2 ? 1 : 0;
        return 0;
    }
    const double axis = paged_tc_axis(a);
    if (axis * 1024 > 4e18) return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    a.grid = axis / 1024 < a.n_sm ? static_cast<int>(axis / 1024) + 1 : a.n_sm;
    if (a.grid > 1023) a.grid = 1023;
    return a.grid * 32LL + 2LL * a.grid * a.slot_rows * (a.D + 2) * 4;
}

static int paged_shape_ok(const char *who, int T, int n_seq, int H, int H_kv, int D, int max_pages, int P, int dtype) {
    if (T < 0 || n_seq < 0 || H < 1 || max_pages < 0)
        return fail(ATTN_EINVAL, "%s: need T >= 0, n_seq >= 0, H >= 1, max_pages >= 0", who);
    if (H_kv < 1 || H % H_kv != 0)
        return fail(ATTN_EINVAL, "%s: H_kv must divide H (got H = %d, H_kv = %d)", who, H, H_kv);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, D);
    if (P < 1) return fail(ATTN_EINVAL, "%s: a page must have rows (got %d)", who, P);
    if (P % 8) return fail(ATTN_EUNSUPPORTED, "%s: pages of %d rows not supported (a multiple of 8)", who, P);
    if (static_cast<long long>(max_pages) * P > 0x7fffffffLL)
        return fail(ATTN_EINVAL, "%s: %d pages of %d rows are too many for a sequence", who, max_pages, P);
    return ATTN_OK;
}

ATTN_API long long attn_fwd_paged_workspace(int T, int n_seq, int H, int H_kv, int D, int max_pages, int page_size, int ragged,
                                            int dtype) {
    int rc = paged_shape_ok("attn_fwd_paged_workspace", T, n_seq, H, H_kv, D, max_pages, page_size, dtype);
    if (rc) return rc;
    if (!ragged && n_seq > 0 && T % n_seq) return ATTN_EINVAL;
    PagedArgs a{};
    a.T = T, a.n_seq = n_seq, a.H = H, a.H_kv = H_kv, a.D = D, a.P = page_size, a.max_len = max_pages * page_size;
    return paged_sizes("attn_fwd_paged_workspace", a, ragged != 0, dtype);
}

ATTN_API int attn_fwd_paged(const void *q, const void *kpages, const void *vpages, void *out, float *lse, int T, int H,
                            int H_kv, int D, const long long *strides, int n_pages, int page_size, const int32_t *page_table,
                            int max_pages, long long table_stride, const int32_t *cu_seqlens, const int32_t *cache_len,
                            int n_seq, float scale, int dtype, void *workspace, long long workspace_bytes, void *stream) {
    g_last_error[0] = '\0';
    const char *who = "attn_fwd_paged";
    int rc = paged_shape_ok(who, T, n_seq, H, H_kv, D, max_pages, page_size, dtype);
    if (rc) return rc;
    if (n_pages < 0) return fail(ATTN_EINVAL, "%s: need n_pages >= 0 (got %d)", who, n_pages);
    if (!(scale >= 0.f) || isinf(scale)) return fail(ATTN_EINVAL, "%s: scale must be finite and >= 0", who);
    if (!cu_seqlens && n_seq > 0 && T % n_seq)
        return fail(ATTN_EINVAL, "%s: without cu_seqlens T must be a multiple of n_seq (got %d, %d)", who, T, n_seq);
    if (T == 0 || n_seq == 0) return ATTN_OK;
    if (max_pages == 0) n_pages = 0;  // nothing is read
    if (max_pages > 0 && n_pages == 0) return fail(ATTN_EINVAL, "%s: a table of pages needs n_pages >= 1", who);
    if (!q || !out || (n_pages > 0 && (!kpages || !vpages || !page_table))) return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (!aligned16(q) || !aligned16(out) || (n_pages > 0 && (!aligned16(kpages) || !aligned16(vpages))))
        return fail(ATTN_EINVAL, "%s: q, kpages, vpages and out must be 16-byte aligned", who);
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(cu_seqlens) |
         reinterpret_cast<uintptr_t>(cache_len) | reinterpret_cast<uintptr_t>(lse)) & 3u)
        return fail(ATTN_EINVAL, "%s: page_table, cu_seqlens, cache_len and lse must be 4-byte aligned", who);
    if (n_seq > 1 && (table_stride < 0 || table_stride > kMaxStride / n_seq))
        return fail(ATTN_EINVAL, "%s: table_stride %lld is negative or too large", who, table_stride);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    const long long dense[4] = {static_cast<long long>(H) * D, D, static_cast<long long>(H) * D, D};
    const long long *st = strides ? strides : dense;
    const Rows rq = make_rows(q, T, H, st[0], st[1], D, esz), ro = make_rows(out, T, H, st[2], st[3], D, esz);
    const Rows *rows[2] = {&rq, &ro};
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "out" : "q";
        if (!rows_distinct(*rows[i]) || rows[i]->so >= (1LL << 40) || rows[i]->si >= (1LL << 40))
            return fail(ATTN_EINVAL, "%s: the rows of %s overlap or lie too far apart", who, name);
        if (rows[i]->so % 16 || rows[i]->si % 16)
            return fail(ATTN_EINVAL, "%s: the strides of %s must be multiples of 16 bytes", who, name);
    }
    Pool pool[2];
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "vpages" : "kpages";
        if (!make_pool(&pool[i], i ? vpages : kpages, 1, 0, n_pages, H_kv, page_size, D, esz, strides ? strides + 4 + 3 * i : nullptr))
            return fail(ATTN_EINVAL, "%s: a stride of %s is negative or too large", who, name);
        for (int x = 1; x < 4; ++x)
            if (pool[i].st[x] % 16 || pool[i].st[x] >= (1LL << 40))
                return fail(ATTN_EINVAL, "%s: the strides of %s must be multiples of 16 bytes, below 2^40", who, name);
        if (overlaps(out, static_cast<size_t>((ro.n_outer - 1) * ro.so + (ro.n_inner - 1) * ro.si + ro.row), pool[i].p,
                     pool_extent(pool[i])))
            return fail(ATTN_EINVAL, "%s: out overlaps %s", who, name);
    }
    if (rows_overlap(ro, rq)) return fail(ATTN_EINVAL, "%s: out overlaps q", who);
    const Index index[3] = {table_index(page_table, n_pages, n_seq, max_pages, table_stride),
                            {cu_seqlens, n_seq + 1LL, "cu_seqlens"}, {cache_len, n_seq, "cache_len"}};
    const Rows lr = make_rows(lse, T, 1, H, H, H, 4);
    if (lse && (rows_overlap(lr, rq) || rows_overlap(lr, ro) ||
                overlaps(lse, static_cast<size_t>(T) * H * 4, pool[0].p, pool_extent(pool[0])) ||
                overlaps(lse, static_cast<size_t>(T) * H * 4, pool[1].p, pool_extent(pool[1]))))
        return fail(ATTN_EINVAL, "%s: lse overlaps another tensor", who);
    if (const char *name = index_under(ro, index)) return fail(ATTN_EINVAL, "%s: out overlaps %s", who, name);
    if (const char *name = index_under(lr, index)) return fail(ATTN_EINVAL, "%s: lse overlaps %s", who, name);
    PagedArgs a{};
    a.T = T, a.n_seq = n_seq, a.H = H, a.H_kv = H_kv, a.D = D, a.P = page_size, a.n_pages = n_pages;
    a.max_len = max_pages * page_size;
    const long long need = paged_sizes(who, a, cu_seqlens != nullptr, dtype);
    if (need < 0) return static_cast<int>(need);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned16(workspace))
            return fail(ATTN_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes (got %lld)", who, need,
                        workspace ? workspace_bytes : 0LL);
        const Rows wr = make_rows(workspace, 1, 1, need, need, need, 1);
        const size_t nb = static_cast<size_t>(need);
        if (rows_overlap(wr, rq) || rows_overlap(wr, ro) || (lse && rows_overlap(wr, lr)) ||
            overlaps(workspace, nb, pool[0].p, pool_extent(pool[0])) || overlaps(workspace, nb, pool[1].p, pool_extent(pool[1])) ||
            index_under(wr, index))
            return fail(ATTN_EINVAL, "%s: workspace overlaps a tensor", who);
    }
    int *status = nullptr;
    if ((rc = status_word(&status))) return rc;
    a.q = q, a.k = kpages, a.v = vpages, a.out = out, a.lse = lse;
    a.page_table = page_table, a.cu_seqlens = cu_seqlens, a.cache_len = cache_len;
    a.table_stride = n_seq > 1 ? table_stride : 0;
    a.q_ts = rq.so / esz, a.q_hs = rq.si / esz, a.o_ts = ro.so / esz, a.o_hs = ro.si / esz;
    a.k_ps = pool[0].st[1] / esz, a.k_hs = pool[0].st[2] / esz, a.k_rs = pool[0].st[3] / esz;
    a.v_ps = pool[1].st[1] / esz, a.v_hs = pool[1].st[2] / esz, a.v_rs = pool[1].st[3] / esz;
    a.scale = scale, a.status = status, a.stream = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == ATTN_F32) {
        if (need > 0) {
            a.part_o = static_cast<float *>(workspace);
            a.part_ml = a.part_o + need / 4 / (D + 2) * D;
        }
        e = launch_paged_f32(a);
    } else {
        const long long parts = 2LL * a.grid * a.slot_rows;
        if (need > 0) {
            a.part_o = static_cast<float *>(workspace);
            a.part_ml = a.part_o + parts * D;
            a.merge = reinterpret_cast<int *>(a.part_ml + parts * 2);
        }
        CUtensorMap tq, tk, tv;
        if (n_pages == 0)  // no box is copied: any valid view
            for (int i = 0; i < 2; ++i) make_pool(&pool[i], q, 1, 0, 1, 1, page_size, D, esz, nullptr);
        Heads heads[2] = {};
        a.halves = !even_heads(pool[0], &heads[0]) || !even_heads(pool[1], &heads[1]);
        if (a.halves) a.box = 8;
        a.k_pstep = static_cast<int>(heads[0].pstep), a.k_hstep = static_cast<int>(heads[0].hstep);
        a.v_pstep = static_cast<int>(heads[1].pstep), a.v_hstep = static_cast<int>(heads[1].hstep);
        if ((rc = make_map_tokens(&tq, rq, D, a.heads, a.box_tokens)) ||
            (rc = make_map_pages(&tk, pool[0], a.halves ? nullptr : &heads[0], a.box)) ||
            (rc = make_map_pages(&tv, pool[1], a.halves ? nullptr : &heads[1], a.box)))
            return rc;
        e = launch_paged_tc(a, tq, tk, tv);
    }
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_fwd_paged launch");
}

// Shared by attn_rope (no cache) and attn_rope_append.
static int rope_impl(const char *who, RopeArgs a, const long long *strides, const double *freqs, int inverse,
                     int dtype, void *stream) {
    g_last_error[0] = '\0';
    const bool append = a.append != 0;
    if (a.T < 0 || a.H < 1 || a.H_kv < 0 || (append && (a.H_kv < 1 || a.B < 1 || a.Skv < 0)))
        return fail(ATTN_EINVAL, "%s: need T >= 0, H >= 1, H_kv >= %d%s", who, append ? 1 : 0,
                    append ? ", B >= 1, Skv >= 0" : "");
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (a.D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, a.D);
    if (a.D != 64 && a.D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, a.D);
    if (a.rotary_dim < 0 || a.rotary_dim > a.D || a.rotary_dim % 2)
        return fail(ATTN_EINVAL, "%s: rotary_dim must be even, in [0, D] (got %d)", who, a.rotary_dim);
    if ((a.interleaved != 0 && a.interleaved != 1) || (inverse != 0 && inverse != 1))
        return fail(ATTN_EINVAL, "%s: interleaved and inverse must be 0 or 1", who);
    if (!(fabsf(a.mscale) <= 3.4e38f)) return fail(ATTN_EINVAL, "%s: mscale must be finite", who);
    if (a.rotary_dim > 0 && !freqs) return fail(ATTN_EINVAL, "%s: freqs must not be NULL", who);
    for (int p = 0; p < a.rotary_dim / 2; ++p)
        if (!isfinite(freqs[p])) return fail(ATTN_EINVAL, "%s: freqs[%d] is not finite", who, p);
    if (a.T == 0) return ATTN_OK;
    if (!a.q || !a.q_out || (a.H_kv > 0 && !a.k) || (!append && a.H_kv > 0 && !a.k_out) ||
        (append && (!a.v || (a.Skv > 0 && (!a.kcache || !a.vcache)))))
        return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (!append && !a.positions) return fail(ATTN_EINVAL, "%s: positions must not be NULL", who);
    if (append && !a.cu_seqlens && a.T % a.B)
        return fail(ATTN_EINVAL, "%s: without cu_seqlens T must be a multiple of B (got %d, %d)", who, a.T, a.B);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    const uintptr_t amask = static_cast<uintptr_t>(esz - 1);
    if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
         reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out)) & amask)
        return fail(ATTN_EINVAL, "%s: tensors must be aligned to their element size", who);
    if (!aligned16(a.kcache) || !aligned16(a.vcache))
        return fail(ATTN_EINVAL, "%s: kcache and vcache must be 16-byte aligned", who);
    if ((reinterpret_cast<uintptr_t>(a.cu_seqlens) | reinterpret_cast<uintptr_t>(a.cache_len) |
         reinterpret_cast<uintptr_t>(a.positions)) & 3u)
        return fail(ATTN_EINVAL, "%s: cu_seqlens, cache_len and positions must be 4-byte aligned", who);
    // views: q, k, v, q_out, k_out
    const void *ptrs[5] = {a.q, a.H_kv ? a.k : nullptr, append ? a.v : nullptr, a.q_out, a.H_kv ? a.k_out : nullptr};
    const int heads[5] = {a.H, a.H_kv, a.H_kv, a.H, a.H_kv};
    const char *names[5] = {"q", "k", "v", "q_out", "k_out"};
    const long long vec = 16 / esz;
    Rows rows[5];
    long long st[5][2];
    bool wide = (a.rotary_dim / 2) % vec == 0;
    for (int i = 0; i < 5; ++i) {
        st[i][0] = strides ? strides[2 * i] : static_cast<long long>(heads[i]) * a.D;
        st[i][1] = strides ? strides[2 * i + 1] : a.D;
        rows[i] = make_rows(ptrs[i], a.T, heads[i], st[i][0], st[i][1], a.D, esz);
        if (!ptrs[i]) continue;
        if (!rows_distinct(rows[i]))
            return fail(ATTN_EINVAL, "%s: the rows of %s overlap (strides %lld, %lld)", who, names[i], st[i][0], st[i][1]);
        st[i][0] = rows[i].so / esz;
        st[i][1] = rows[i].si / esz;
        wide = wide && aligned16(ptrs[i]) && st[i][0] % vec == 0 && st[i][1] % vec == 0;
    }
    // an output may be its own input (in place); any other overlap is an error
    for (int o = 3; o < 5; ++o)
        for (int i = 0; i < 5; ++i) {
            if (i == o || (i < 3 && i == o - 3 && same_rows(rows[i], rows[o]))) continue;
            if (rows_overlap(rows[o], rows[i])) return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, names[o], names[i]);
        }
    if (append) {
        const long long cache_rows = static_cast<long long>(a.B) * a.H_kv;
        const long long head = static_cast<long long>(a.Skv) * a.D;
        const Rows kc = make_rows(a.kcache, cache_rows, 1, head, head, head, esz);
        const Rows vc = make_rows(a.vcache, cache_rows, 1, head, head, head, esz);
        if (a.Skv > 0) {
            if (rows_overlap(kc, vc)) return fail(ATTN_EINVAL, "%s: kcache overlaps vcache", who);
            for (int i = 0; i < 5; ++i)
                if (rows_overlap(kc, rows[i]) || rows_overlap(vc, rows[i]))
                    return fail(ATTN_EINVAL, "%s: %s overlaps a cache", who, names[i]);
        }
    }
    a.q_ts = st[0][0], a.q_hs = st[0][1], a.k_ts = st[1][0], a.k_hs = st[1][1], a.v_ts = st[2][0], a.v_hs = st[2][1];
    a.qo_ts = st[3][0], a.qo_hs = st[3][1], a.ko_ts = st[4][0], a.ko_hs = st[4][1];
    for (int p = 0; p < a.rotary_dim / 2; ++p) a.turns[p] = rope_turns(freqs[p]);
    a.sin_scale = inverse ? -a.mscale : a.mscale;
    a.n_sm = num_sms();
    a.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_rope(a, dtype == ATTN_F32, wide);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, who);
}

ATTN_API int attn_rope(const void *q, const void *k, void *q_out, void *k_out, int T, int H, int H_kv, int D,
                       const long long *strides, const int32_t *positions, const double *freqs, int rotary_dim,
                       int interleaved, int inverse, float mscale, int dtype, void *stream) {
    RopeArgs a{};
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
    a.T = T, a.H = H, a.H_kv = H_kv, a.D = D;
    a.positions = positions;
    a.rotary_dim = rotary_dim, a.interleaved = interleaved, a.mscale = mscale;
    // strides holds q, k, q_out, k_out; rope_impl takes q, k, v, q_out, k_out
    long long st[10] = {};
    if (strides) {
        for (int i = 0; i < 4; ++i) st[i] = strides[i];
        for (int i = 0; i < 4; ++i) st[6 + i] = strides[4 + i];
    }
    return rope_impl("attn_rope", a, strides ? st : nullptr, freqs, inverse, dtype, stream);
}

ATTN_API int attn_rope_append(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *kcache,
                              void *vcache, int T, int H, int H_kv, int D, const long long *strides, int B, int Skv,
                              const int32_t *cu_seqlens, const int32_t *cache_len, const int32_t *positions,
                              const double *freqs, int rotary_dim, int interleaved, float mscale, int dtype,
                              void *stream) {
    RopeArgs a{};
    a.append = 1;
    a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.k_out = k_out, a.kcache = kcache, a.vcache = vcache;
    a.T = T, a.H = H, a.H_kv = H_kv, a.D = D, a.B = B, a.Skv = Skv;
    a.cu_seqlens = cu_seqlens, a.cache_len = cache_len, a.positions = positions;
    a.rotary_dim = rotary_dim, a.interleaved = interleaved, a.mscale = mscale;
    return rope_impl("attn_rope_append", a, strides, freqs, 0, dtype, stream);
}

// Shared by attn_norm_rope (no cache) and attn_rope_append_paged.  strides: q, k, v,
// q_out, k_out (token, head), kpages, vpages (page, head, row), or NULL.
static int norm_rope_impl(const char *who, NormRopeArgs a, const long long *strides, const double *freqs, int max_pages,
                          int dtype, void *stream) {
    g_last_error[0] = '\0';
    const bool append = a.append != 0;
    if (a.T < 0 || a.H < 1 || a.H_kv < 0 || (append && (a.H_kv < 1 || a.n_seq < 0 || max_pages < 0 || a.n_pages < 0)))
        return fail(ATTN_EINVAL, "%s: need T >= 0, H >= 1, H_kv >= %d%s", who, append ? 1 : 0,
                    append ? ", n_seq >= 0, max_pages >= 0, n_pages >= 0" : "");
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (a.D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, a.D);
    if (a.D != 64 && a.D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, a.D);
    if (a.rotary_dim < 0 || a.rotary_dim > a.D || a.rotary_dim % 2)
        return fail(ATTN_EINVAL, "%s: rotary_dim must be even, in [0, D] (got %d)", who, a.rotary_dim);
    if (a.interleaved != 0 && a.interleaved != 1) return fail(ATTN_EINVAL, "%s: interleaved must be 0 or 1", who);
    if (!(fabsf(a.mscale) <= 3.4e38f)) return fail(ATTN_EINVAL, "%s: mscale must be finite", who);
    if (!(a.eps >= 0.f && a.eps <= 3.4e38f)) return fail(ATTN_EINVAL, "%s: eps must be finite and >= 0", who);
    if (a.rotary_dim > 0 && !freqs) return fail(ATTN_EINVAL, "%s: freqs must not be NULL", who);
    for (int p = 0; p < a.rotary_dim / 2; ++p)
        if (!isfinite(freqs[p])) return fail(ATTN_EINVAL, "%s: freqs[%d] is not finite", who, p);
    if (append && a.P < 1) return fail(ATTN_EINVAL, "%s: a page must have rows (got %d)", who, a.P);
    if (append && static_cast<long long>(max_pages) * a.P > 0x7fffffffLL)
        return fail(ATTN_EINVAL, "%s: %d pages of %d rows are too many for a sequence", who, max_pages, a.P);
    if (a.T == 0 || (append && a.n_seq == 0)) return ATTN_OK;
    if (append && max_pages == 0) a.n_pages = 0;  // every token is turned, none cached
    a.max_len = append ? max_pages * a.P : 0;
    if (append && max_pages > 0 && a.n_pages == 0) return fail(ATTN_EINVAL, "%s: a table of pages needs n_pages >= 1", who);
    if (!a.q || !a.q_out || (a.H_kv > 0 && !a.k) || (!append && a.H_kv > 0 && !a.k_out) ||
        (append && (!a.v || (a.n_pages > 0 && (!a.kpages || !a.vpages || !a.page_table)))))
        return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (!append && !a.positions) return fail(ATTN_EINVAL, "%s: positions must not be NULL", who);
    if (append && !a.cu_seqlens && a.T % a.n_seq)
        return fail(ATTN_EINVAL, "%s: without cu_seqlens T must be a multiple of n_seq (got %d, %d)", who, a.T, a.n_seq);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    const uintptr_t amask = static_cast<uintptr_t>(esz - 1);
    if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
         reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.kpages) |
         reinterpret_cast<uintptr_t>(a.vpages) | reinterpret_cast<uintptr_t>(a.q_weight) |
         reinterpret_cast<uintptr_t>(a.k_weight)) & amask)
        return fail(ATTN_EINVAL, "%s: tensors must be aligned to their element size", who);
    if ((reinterpret_cast<uintptr_t>(a.cu_seqlens) | reinterpret_cast<uintptr_t>(a.cache_len) |
         reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.page_table)) & 3u)
        return fail(ATTN_EINVAL, "%s: cu_seqlens, cache_len, positions and page_table must be 4-byte aligned", who);
    if (append && a.n_seq > 1 && (a.table_stride < 0 || a.table_stride > kMaxStride / a.n_seq))
        return fail(ATTN_EINVAL, "%s: table_stride %lld is negative or too large", who, a.table_stride);
    // views: q, k, v, q_out, k_out
    const void *ptrs[5] = {a.q, a.H_kv ? a.k : nullptr, append ? a.v : nullptr, a.q_out, a.H_kv ? a.k_out : nullptr};
    const int heads[5] = {a.H, a.H_kv, a.H_kv, a.H, a.H_kv};
    const char *names[5] = {"q", "k", "v", "q_out", "k_out"};
    const long long vec = 16 / esz;
    Rows rows[5];
    long long st[5][2];
    // pairs side by side need whole units only, halves also whole units of pairs
    bool wide = (a.interleaved || (a.rotary_dim / 2) % vec == 0) && aligned16(a.q_weight) && aligned16(a.k_weight);
    for (int i = 0; i < 5; ++i) {
        st[i][0] = strides ? strides[2 * i] : static_cast<long long>(heads[i]) * a.D;
        st[i][1] = strides ? strides[2 * i + 1] : a.D;
        rows[i] = make_rows(ptrs[i], a.T, heads[i], st[i][0], st[i][1], a.D, esz);
        if (!ptrs[i]) continue;
        if (!rows_distinct(rows[i]))
            return fail(ATTN_EINVAL, "%s: the rows of %s overlap (strides %lld, %lld)", who, names[i], st[i][0], st[i][1]);
        st[i][0] = rows[i].so / esz;
        st[i][1] = rows[i].si / esz;
        wide = wide && aligned16(ptrs[i]) && st[i][0] % vec == 0 && st[i][1] % vec == 0;
    }
    // an output may be its own input (in place); any other overlap is an error
    for (int o = 3; o < 5; ++o) {
        for (int i = 0; i < 5; ++i) {
            if (i == o || (i < 3 && i == o - 3 && same_rows(rows[i], rows[o]))) continue;
            if (rows_overlap(rows[o], rows[i])) return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, names[o], names[i]);
        }
        for (const void *w : {a.q_weight, a.k_weight})
            if (w && rows_overlap(rows[o], make_rows(w, 1, 1, a.D, a.D, a.D, esz)))
                return fail(ATTN_EINVAL, "%s: %s overlaps a weight", who, names[o]);
    }
    const Index index[4] = {{a.positions, a.T, "positions"},
                            table_index(append ? a.page_table : nullptr, a.n_pages, a.n_seq, max_pages, a.table_stride),
                            {append ? a.cu_seqlens : nullptr, a.n_seq + 1LL, "cu_seqlens"},
                            {append ? a.cache_len : nullptr, a.n_seq, "cache_len"}};
    for (int o = 3; o < 5; ++o)
        if (const char *name = index_under(rows[o], index)) return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, names[o], name);
    if (append) {
        Pool pool[2];
        for (int i = 0; i < 2; ++i) {
            const char *name = i ? "vpages" : "kpages";
            if (!make_pool(&pool[i], i ? a.vpages : a.kpages, 1, 0, a.n_pages, a.H_kv, a.P, a.D, esz,
                           strides ? strides + 10 + 3 * i : nullptr))
                return fail(ATTN_EINVAL, "%s: a stride of %s is negative or too large", who, name);
            if (!pool_distinct(pool[i])) return fail(ATTN_EINVAL, "%s: the rows of %s overlap", who, name);
            const Rows pr = make_rows(pool[i].p, 1, 1, 1, 1, static_cast<long long>(pool_extent(pool[i])), 1);
            for (int x = 0; x < 5; ++x)
                if (!pool_empty(pool[i]) && rows_overlap(pr, rows[x]))
                    return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, names[x], name);
            if (const char *under = pool_empty(pool[i]) ? nullptr : index_under(pr, index))
                return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, name, under);
            if (!pool_empty(pool[i]) &&
                ((a.q_weight && overlaps(a.q_weight, static_cast<size_t>(a.D * esz), pool[i].p, pool_extent(pool[i]))) ||
                 (a.k_weight && overlaps(a.k_weight, static_cast<size_t>(a.D * esz), pool[i].p, pool_extent(pool[i])))))
                return fail(ATTN_EINVAL, "%s: a weight overlaps %s", who, name);
            if (!pool_empty(pool[i]))
                wide = wide && aligned16(pool[i].p) && pool[i].st[1] % 16 == 0 && pool[i].st[2] % 16 == 0 && pool[i].st[3] % 16 == 0;
        }
        if (pools_overlap(pool[0], pool[1])) return fail(ATTN_EINVAL, "%s: kpages overlaps vpages", who);
        a.k_ps = pool[0].st[1] / esz, a.k_hs = pool[0].st[2] / esz, a.k_rs = pool[0].st[3] / esz;
        a.v_ps = pool[1].st[1] / esz, a.v_hs = pool[1].st[2] / esz, a.v_rs = pool[1].st[3] / esz;
        if (a.n_seq == 1) a.table_stride = 0;
    }
    a.q_ts = st[0][0], a.q_hs = st[0][1], a.k_ts = st[1][0], a.kt_hs = st[1][1], a.v_ts = st[2][0], a.vt_hs = st[2][1];
    a.qo_ts = st[3][0], a.qo_hs = st[3][1], a.ko_ts = st[4][0], a.ko_hs = st[4][1];
    for (int p = 0; p < a.rotary_dim / 2; ++p) a.turns[p] = rope_turns(freqs[p]);
    a.n_sm = num_sms();
    a.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_norm_rope(a, dtype == ATTN_F32, wide);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, who);
}

ATTN_API int attn_norm_rope(const void *q, const void *k, void *q_out, void *k_out, int T, int H, int H_kv, int D,
                            const long long *strides, const int32_t *positions, const double *freqs, int rotary_dim,
                            int interleaved, float mscale, const void *q_weight, const void *k_weight, float eps, int dtype,
                            void *stream) {
    NormRopeArgs a{};
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out, a.q_weight = q_weight, a.k_weight = k_weight;
    a.T = T, a.H = H, a.H_kv = H_kv, a.D = D, a.positions = positions;
    a.rotary_dim = rotary_dim, a.interleaved = interleaved, a.mscale = mscale, a.eps = eps;
    // strides holds q, k, q_out, k_out; norm_rope_impl takes v between them
    long long st[16] = {};
    if (strides) {
        for (int i = 0; i < 4; ++i) st[i] = strides[i];
        for (int i = 0; i < 4; ++i) st[6 + i] = strides[4 + i];
    }
    return norm_rope_impl("attn_norm_rope", a, strides ? st : nullptr, freqs, 0, dtype, stream);
}

ATTN_API int attn_rope_append_paged(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *kpages,
                                    void *vpages, int T, int H, int H_kv, int D, const long long *strides, int n_pages,
                                    int page_size, const int32_t *page_table, int max_pages, long long table_stride,
                                    const int32_t *cu_seqlens, const int32_t *cache_len, int n_seq, const int32_t *positions,
                                    const double *freqs, int rotary_dim, int interleaved, float mscale, const void *q_weight,
                                    const void *k_weight, float eps, int dtype, void *stream) {
    NormRopeArgs a{};
    a.append = 1;
    a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.k_out = k_out, a.kpages = kpages, a.vpages = vpages;
    a.q_weight = q_weight, a.k_weight = k_weight;
    a.T = T, a.H = H, a.H_kv = H_kv, a.D = D, a.n_pages = n_pages, a.P = page_size, a.n_seq = n_seq;
    a.page_table = page_table, a.table_stride = table_stride;
    a.cu_seqlens = cu_seqlens, a.cache_len = cache_len, a.positions = positions;
    a.rotary_dim = rotary_dim, a.interleaved = interleaved, a.mscale = mscale, a.eps = eps;
    return norm_rope_impl("attn_rope_append_paged", a, strides, freqs, max_pages, dtype, stream);
}

// ------------------------------------------------------------ the table of pages

static long long pages_workspace(int n_out, int n_pages) {
    // held, pins; first or move; need, stays, lost; the list with its count in front
    const long long words = (static_cast<long long>(n_pages) + 31) / 32;
    return (2 * words + n_pages + 3LL * n_out + n_pages + 1) * 4;
}

ATTN_API long long attn_pages_workspace(int n_out, int n_pages) {
    return n_out < 0 || n_pages < 0 ? ATTN_EINVAL : pages_workspace(n_out, n_pages);
}

// Rows of a new table and pairs of a list of copies: the kernels count three entries of each in
// 32 bits.
constexpr int kMaxCopies = 1 << 29;

// Shared by attn_pages_step and attn_pages_compact.
static int pages_impl(const char *who, PagesArgs a, bool step, void *workspace, long long workspace_bytes, void *stream) {
    g_last_error[0] = '\0';
    if (a.n_seq < 0 || a.n_out < 0 || a.max_pages < 0 || a.n_pages < 0)
        return fail(ATTN_EINVAL, "%s: the numbers of sequences and pages must not be negative", who);
    if (a.P < 1) return fail(ATTN_EINVAL, "%s: a page must have rows (got %d)", who, a.P);
    if (static_cast<long long>(a.max_pages) * a.P > 0x7fffffffLL)
        return fail(ATTN_EINVAL, "%s: %d pages of %d rows are too many for a sequence", who, a.max_pages, a.P);
    if (!a.parents && a.n_out != a.n_seq)
        return fail(ATTN_EINVAL, "%s: without parents there are as many rows as before (got %d, %d)", who, a.n_out, a.n_seq);
    // ranks, counts and places in the lists are kept in 32 bits; few entries a row do not bound the rows
    if (static_cast<long long>(a.n_out) * a.max_pages >= (1LL << 30) || a.n_pages >= 1 << 30 || a.n_out > kMaxCopies)
        return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    const bool entries = a.n_seq > 0 && a.max_pages > 0, out_entries = a.n_out > 0 && a.max_pages > 0;
    if (!a.free_pages || (entries && !a.table) || (out_entries && !a.table_out) || (step && a.n_out > 0 && !a.len_out) ||
        (a.n_copies > 0 && !a.copies))
        return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    if (a.n_seq > 1 && (a.table_stride < 0 || a.table_stride > kMaxStride / a.n_seq))
        return fail(ATTN_EINVAL, "%s: table_stride %lld is negative or too large", who, a.table_stride);
    if (a.n_out > 1 && (a.out_stride < a.max_pages || a.out_stride > kMaxStride / a.n_out))
        return fail(ATTN_EINVAL, "%s: out_stride %lld is below max_pages or too large", who, a.out_stride);
    if (a.n_seq <= 1) a.table_stride = 0;
    if (a.n_out <= 1) a.out_stride = 0;
    const long long need = pages_workspace(a.n_out, a.n_pages);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return fail(ATTN_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes (got %lld)", who, need,
                    workspace ? workspace_bytes : 0LL);
    const struct {
        const void *p;
        long long n;
        const char *name;
    } t[] = {
        {a.table_out, out_entries ? (a.n_out - 1) * a.out_stride + a.max_pages : 0, "the new table"},
        {a.len_out, a.n_out, "the new lengths"},
        {a.copies, 3LL * a.n_copies, "copies"},
        {a.free_pages, 1, "free_pages"},
        {workspace, need / 4, "workspace"},
        {a.table, entries ? (a.n_seq - 1) * a.table_stride + a.max_pages : 0, "page_table"},
        {a.cache_len, a.n_seq, "cache_len"},
        {a.parents, a.n_out, "parents"},
        {a.new_len, a.n_out, "new_len"},
        {a.pinned, a.n_pages, "pinned"},
    };
    for (int i = 0; i < 10; ++i) {
        if (!t[i].p) continue;
        if (reinterpret_cast<uintptr_t>(t[i].p) & 3u) return fail(ATTN_EINVAL, "%s: %s must be 4-byte aligned", who, t[i].name);
        for (int j = 0; j < i && j < 5; ++j)
            if (t[j].p && overlaps(t[i].p, static_cast<size_t>(t[i].n) * 4, t[j].p, static_cast<size_t>(t[j].n) * 4))
                return fail(ATTN_EINVAL, "%s: %s overlaps %s", who, t[j].name, t[i].name);
    }
    a.words = (a.n_pages + 31) / 32;
    a.held = static_cast<unsigned *>(workspace);
    a.pins = a.held + a.words;
    int32_t *rest = reinterpret_cast<int32_t *>(a.pins + a.words);
    if (step)
        a.first = rest;
    else
        a.move = rest;
    a.need = rest + a.n_pages;
    a.stays = a.need + a.n_out;
    a.lost = a.stays + a.n_out;
    a.list = a.lost + a.n_out + 1;
    a.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = step ? launch_pages_step(a) : launch_pages_compact(a);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, who);
}

ATTN_API int attn_pages_step(const int32_t *page_table, const int32_t *cache_len, int n_seq, int max_pages, long long table_stride,
                             int n_pages, int page_size, const int32_t *parents, const int32_t *new_len,
                             const int32_t *pinned, int n_out, int32_t *table_out, long long out_stride, int32_t *len_out,
                             int32_t *copies, int32_t *free_pages, void *workspace, long long workspace_bytes,
                             void *stream) {
    PagesArgs a{};
    a.table = page_table, a.cache_len = cache_len, a.parents = parents, a.new_len = new_len, a.pinned = pinned;
    a.table_out = table_out, a.len_out = len_out, a.copies = copies, a.free_pages = free_pages;
    a.table_stride = table_stride, a.out_stride = out_stride;
    a.n_seq = n_seq, a.n_out = n_out, a.max_pages = max_pages, a.P = page_size, a.n_pages = n_pages, a.n_copies = n_out;
    return pages_impl("attn_pages_step", a, true, workspace, workspace_bytes, stream);
}

ATTN_API int attn_pages_compact(const int32_t *page_table, const int32_t *cache_len, int n_seq, int max_pages,
                                long long table_stride, int n_pages, int page_size, const int32_t *pinned, int32_t *table_out,
                                long long out_stride, int32_t *copies, int32_t *free_pages, void *workspace,
                                long long workspace_bytes, void *stream) {
    PagesArgs a{};
    a.table = page_table, a.cache_len = cache_len, a.pinned = pinned;
    a.table_out = table_out, a.copies = copies, a.free_pages = free_pages;
    a.table_stride = table_stride, a.out_stride = out_stride;
    a.n_seq = a.n_out = n_seq, a.max_pages = max_pages, a.P = page_size, a.n_pages = n_pages, a.n_copies = (n_pages + 1) / 2;
    return pages_impl("attn_pages_compact", a, false, workspace, workspace_bytes, stream);
}

ATTN_API int attn_pages_copy(void *kpages, void *vpages, int layers, int n_pages, int H_kv, int page_size, int D,
                             const long long *strides, const int32_t *copies, int n_copies, int dtype, void *stream) {
    g_last_error[0] = '\0';
    const char *who = "attn_pages_copy";
    if (layers < 0 || n_pages < 0 || H_kv < 1 || n_copies < 0)
        return fail(ATTN_EINVAL, "%s: need layers >= 0, n_pages >= 0, H_kv >= 1, n_copies >= 0", who);
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return fail(ATTN_EINVAL, "%s: unknown dtype %d", who, dtype);
    if (D <= 0) return fail(ATTN_EINVAL, "%s: D must be positive (got %d)", who, D);
    if (D != 64 && D != 128) return fail(ATTN_EUNSUPPORTED, "%s: D = %d not supported (64 or 128)", who, D);
    if (page_size < 1) return fail(ATTN_EINVAL, "%s: a page must have rows (got %d)", who, page_size);
    if (static_cast<long long>(H_kv) * page_size >= (1LL << 30) || layers >= 1 << 30 || n_copies > kMaxCopies)
        return fail(ATTN_EINVAL, "%s: the sizes are too large", who);
    if (layers == 0 || n_pages == 0 || n_copies == 0) return ATTN_OK;
    if (!kpages || !vpages || !copies) return fail(ATTN_EINVAL, "%s: a tensor is NULL", who);
    const long long esz = dtype == ATTN_BF16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(kpages) | reinterpret_cast<uintptr_t>(vpages)) & static_cast<uintptr_t>(esz - 1))
        return fail(ATTN_EINVAL, "%s: tensors must be aligned to their element size", who);
    if (reinterpret_cast<uintptr_t>(copies) & 3u) return fail(ATTN_EINVAL, "%s: copies must be 4-byte aligned", who);
    Pool pool[2];
    bool wide = true;
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "vpages" : "kpages";
        if (!make_pool(&pool[i], i ? vpages : kpages, layers, strides ? strides[4 * i] : 0, n_pages, H_kv, page_size, D, esz,
                       strides ? strides + 4 * i + 1 : nullptr))
            return fail(ATTN_EINVAL, "%s: a stride of %s is negative or too large", who, name);
        if (!pool_distinct(pool[i])) return fail(ATTN_EINVAL, "%s: the rows of %s overlap", who, name);
        if (overlaps(copies, static_cast<size_t>(n_copies) * 12, pool[i].p, pool_extent(pool[i])))
            return fail(ATTN_EINVAL, "%s: copies overlaps %s", who, name);
        wide = wide && aligned16(pool[i].p);
        for (int x = 0; x < 4; ++x) wide = wide && pool[i].st[x] % 16 == 0;
    }
    if (pools_overlap(pool[0], pool[1])) return fail(ATTN_EINVAL, "%s: kpages overlaps vpages", who);
    PagesCopyArgs a{};
    a.k = {const_cast<char *>(pool[0].p), pool[0].st[0], pool[0].st[1], pool[0].st[2], pool[0].st[3]};
    a.v = {const_cast<char *>(pool[1].p), pool[1].st[0], pool[1].st[1], pool[1].st[2], pool[1].st[3]};
    a.copies = copies, a.n_copies = n_copies, a.layers = layers, a.n_pages = n_pages, a.H_kv = H_kv, a.P = page_size;
    a.row_bytes = static_cast<int>(D * esz);
    a.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_pages_copy(a, wide, static_cast<int>(esz));
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, who);
}

ATTN_API int attn_device_status(void *stream) {
    g_last_error[0] = '\0';
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_device_status: stream synchronize");
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    int word = 0;
    e = cudaMemcpy(&word, status, sizeof word, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "attn_device_status: read status word");
    if (word == 0) return ATTN_OK;
    const int zero = 0;
    e = cudaMemcpy(status, &zero, sizeof zero, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "attn_device_status: clear status word");
    if ((word & 0xff) == kStatusSchedConflict)
        return fail(ATTN_ECONFLICT,
                    "two bf16 prefill launches in flight shared one work counter (site 0x%x); "
                    "their outputs are undefined", word >> 8);
    return fail(ATTN_ETIMEOUT, "a device-side wait gave up (site 0x%x); that call's output is undefined",
                word >> 8);
}

ATTN_API int attn_selftest_wait_timeout(long long limit_cycles, void *stream) {
    g_last_error[0] = '\0';
    if (limit_cycles < 0 || limit_cycles > kWaitLimitCycles)
        return fail(ATTN_EINVAL, "attn_selftest_wait_timeout: limit must be in [0, %lld] cycles", kWaitLimitCycles);
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    cudaError_t e = launch_wait_timeout_probe(limit_cycles, status, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "attn_selftest_wait_timeout launch");
}

ATTN_API void attn_release(void) {
    int dev;
    if (current_device(&dev)) return;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        Workspace &w = g_ws[dev];
        if (w.ptr) cudaFree(w.ptr);
        for (int i = 0; i < w.n_retired; ++i) cudaFree(w.retired[i]);
        w.ptr = nullptr;
        w.bytes = 0;
        w.n_retired = 0;
    }
    // outside g_mutex: attn_fwd_host takes its own lock first, then g_mutex
    g_host[dev].release();
    // work counters that a conflict (ATTN_ECONFLICT) may have left unbalanced
    reset_prefill_counters();
}

}  // extern "C"

namespace attn {

namespace {
// Waits on an mbarrier phase that nothing completes, with a short limit, so
// that the timeout path (abort flag, status word) runs without a hang.
__global__ void wait_timeout_probe_kernel(long long limit, int *status) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !mbar_wait(&bar, 0, &abort_flag, limit)) report_timeout(status, 0x7f);
    __syncthreads();
    if (threadIdx.x == 0) mbar_arrive(&bar);  // complete the phase before the CTA exits
}

__global__ void zero_fill_kernel(uint4 *out, size_t n) {
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
         i += static_cast<size_t>(gridDim.x) * blockDim.x)
        out[i] = make_uint4(0, 0, 0, 0);
}
}  // namespace

cudaError_t launch_wait_timeout_probe(long long limit, int *status, cudaStream_t stream) {
    wait_timeout_probe_kernel<<<1, 32, 0, stream>>>(limit, status);
    return cudaGetLastError();
}

cudaError_t launch_zero_fill(void *out, size_t n_bytes, cudaStream_t stream) {
    const size_t n = n_bytes / 16;
    if (n == 0) return cudaSuccess;
    size_t blocks = (n + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    zero_fill_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(static_cast<uint4 *>(out), n);
    return cudaGetLastError();
}

}  // namespace attn
