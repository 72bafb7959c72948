// The table of pages of a paged KV cache, and copies of pages.
//
// attn_pages_step makes the next table from the last one: row b goes on from row
// parents[b], cut back or grown to new_len[b] tokens.  No counts of holders are kept from
// call to call: which pages are held is read off the table, as a set of bits.
//   1. bits = pinned pages; `first` = nobody                     (pages_clear_kernel)
//   2. a warp a row: full pages that stay set their bits (a row that shares a page reads
//      the bit first); a partly filled page takes the lowest row that holds it as such
//                                                                (pages_mark_kernel)
//   3. one block: which rows keep their partly filled page (its first, unless the bit says
//      that another row holds it full or it is pinned), how many new pages each row wants,
//      the prefix sums of both the wants and the free pages of each word of bits, and
//      the list of the lowest free pages, as many as are wanted   (pages_plan_kernel)
//   4. a warp a row: writes it, and the copy it needs             (pages_write_kernel)
// Minima, unions and prefix sums do not depend on the order of the threads, so a call gives
// the same table every time.
//
// attn_pages_compact sets the bits of all pages held (n of them) in the same way; the k-th
// lowest held page from n on moves to the k-th lowest free one below n.
//
// Both move a few hundred KB; what bounds them is the chain of four launches (programmatic
// ones, about 2 us each).  attn_pages_copy moves whole rows of pages, 16 bytes a thread and
// eight in flight, bound by HBM.
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kNobody = 0x7fffffff;

__device__ __forceinline__ bool is_page(const PagesArgs &a, int page) { return page >= 0 && page < a.n_pages; }

__global__ void __launch_bounds__(256) pages_clear_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    for (int w = (blockIdx.x * 256 + threadIdx.x) / 32; w < a.words; w += gridDim.x * 8) {
        const int page = w * 32 + lane;
        const unsigned bits = __ballot_sync(0xffffffffu, a.pinned && page < a.n_pages && a.pinned[page] != 0);
        if (lane == 0) {
            a.held[w] = bits;
            a.pins[w] = bits;
        }
        if (a.first && page < a.n_pages) a.first[page] = kNobody;
    }
}

// What row b keeps of its parent: pages [0, full) whole, `part` rows of the next one.
struct Kept {
    const int32_t *old;
    int full, part, pages;  // pages: that the row is to have
    int len;
};
__device__ __forceinline__ Kept kept_of(const PagesArgs &a, int b) {
    Kept k;
    const int p = a.parents ? a.parents[b] : b;
    const bool some = p >= 0 && p < a.n_seq;
    const int most = a.max_pages * a.P;
    const int L = some ? a.cache_len ? min(max(a.cache_len[p], 0), most) : most : 0;
    k.len = a.new_len ? min(max(a.new_len[b], 0), most) : L;
    const int keep = min(L, k.len);
    k.old = a.table + (some ? p : 0) * a.table_stride;
    k.full = keep / a.P;
    k.part = keep % a.P;
    k.pages = k.len / a.P + (k.len % a.P != 0);
    return k;
}

__global__ void __launch_bounds__(256) pages_mark_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int b = (blockIdx.x * 256 + threadIdx.x) / 32, lane = threadIdx.x % 32;
    if (b >= a.n_out) return;
    const Kept k = kept_of(a, b);
    const int whole = a.first ? k.full : k.full + (k.part != 0);  // compaction: every page alike
    int lost = 0;  // entries that are no pages: asked for anew
    for (int i0 = 0; i0 < whole; i0 += 128) {
        int page[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) page[y] = i0 + 32 * y + lane < whole ? k.old[i0 + 32 * y + lane] : -1;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (i0 + 32 * y + lane >= whole) continue;
            if (!is_page(a, page[y])) {
                ++lost;
                continue;
            }
            const unsigned bit = 1u << (page[y] % 32);
            if (!(*const_cast<volatile unsigned *>(&a.held[page[y] / 32]) & bit)) atomicOr(&a.held[page[y] / 32], bit);
        }
    }
    if (!a.first) return;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) lost += __shfl_xor_sync(0xffffffffu, lost, d);
    if (lane == 0) {
        a.need[b] = lost;
        if (k.part && is_page(a, k.old[k.full])) atomicMin(&a.first[k.old[k.full]], b);
    }
}

// Sum of the values of the threads before this one, and of all of them.  The whole block
// calls it.
__device__ __forceinline__ int block_prefix(int v, int *total) {
    __shared__ int sums[kPlanThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int w = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    __syncthreads();
    return s - v + (warp ? before : 0);
}

__device__ __forceinline__ unsigned pages_of_word(const PagesArgs &a, int w) {  // bits that stand for a page
    const int n = a.n_pages - w * 32;
    return n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x;
    // rows: who keeps its partly filled page, and the wants
    int wants = 0;
    for (int b0 = 0; b0 < a.n_out; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int want = 0;
        if (b < a.n_out) {
            const Kept k = kept_of(a, b);
            int stays = 0;
            if (k.part) {
                const int page = k.old[k.full];
                // a row whose page this is sets the bit below: no other row is its first
                if (is_page(a, page) && a.first[page] == b && !(*const_cast<volatile unsigned *>(&a.held[page / 32]) >> (page % 32) & 1u)) {
                    stays = 1;
                    atomicOr(&a.held[page / 32], 1u << (page % 32));
                }
            }
            want = a.need[b] + k.pages - k.full - stays;
            a.stays[b] = stays;
        }
        int all;
        const int at = wants + block_prefix(want, &all);
        if (b < a.n_out) a.need[b] = at;  // the row's first new page in the list
        wants += all;
    }
    __threadfence_block();
    __syncthreads();
    int free_pages = 0;
    for (int w0 = 0; w0 < a.words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        unsigned bits = w < a.words ? ~*const_cast<volatile unsigned *>(&a.held[w]) & pages_of_word(a, w) : 0u;
        int all;
        int at = free_pages + block_prefix(__popc(bits), &all);
        for (; bits && at < wants; ++at) {
            a.list[at] = w * 32 + __ffs(bits) - 1;
            bits &= bits - 1;
        }
        free_pages += all;
    }
    if (tid == 0) {
        a.list[-1] = free_pages;
        *a.free_pages = free_pages - wants;
    }
}

__global__ void __launch_bounds__(256) pages_write_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int b = (blockIdx.x * 256 + threadIdx.x) / 32, lane = threadIdx.x % 32;
    if (b >= a.n_out) return;
    const Kept k = kept_of(a, b);
    const int stays = a.stays[b], n_free = a.list[-1];
    int nth = a.need[b];  // in the list of free pages
    int32_t *out = a.table_out + b * a.out_stride;
    int to = -1;  // the copy of the partly filled page
    for (int i0 = 0; i0 < a.max_pages; i0 += 32) {
        const int i = i0 + lane;
        int page = -1;
        if (i < k.full + stays) page = k.old[i];
        const bool wanted = i < k.pages && (i >= k.full + stays || !is_page(a, page));
        const unsigned all = __ballot_sync(0xffffffffu, wanted);
        const int at = nth + __popc(all & ((1u << lane) - 1u));
        if (wanted) page = at < n_free ? a.list[at] : -1;
        nth += __popc(all);
        if (i < a.max_pages) out[i] = page;
        if (i == k.full) to = page;
    }
    to = __shfl_sync(0xffffffffu, to, k.full % 32);
    if (lane == 0) {
        a.len_out[b] = k.len;
        const int from = k.part ? k.old[k.full] : -1;
        const bool copied = k.part && !stays && is_page(a, from) && to >= 0;
        a.copies[3 * b] = copied ? from : -1;
        a.copies[3 * b + 1] = copied ? to : -1;
        a.copies[3 * b + 2] = copied ? k.part : 0;
    }
}

// Compaction: n pages are held or pinned; lists the free ones below n, then the movable ones
// from n on with the places they go to.
__global__ void __launch_bounds__(kPlanThreads) pages_moves_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x;
    int n = 0;
    for (int w = tid; w < a.words; w += kPlanThreads) n += __popc(a.held[w]);
    int all;
    block_prefix(n, &all);
    n = all;
    int holes = 0, moves = 0;
    for (int w0 = 0; w0 < a.words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        unsigned free_bits = 0, moved = 0;
        if (w < a.words) {
            const unsigned held = a.held[w];
            const unsigned below = n - w * 32 >= 32 ? 0xffffffffu : n > w * 32 ? (1u << (n - w * 32)) - 1u : 0u;  // pages < n
            free_bits = ~held & below;
            moved = held & ~below & ~a.pins[w];
        }
        int at = holes + block_prefix(__popc(free_bits), &all);
        holes += all;
        for (; free_bits; ++at, free_bits &= free_bits - 1) a.list[at] = w * 32 + __ffs(free_bits) - 1;
        at = moves + block_prefix(__popc(moved), &all);
        moves += all;
        for (; moved; ++at, moved &= moved - 1) {
            const int page = w * 32 + __ffs(moved) - 1;
            a.move[page] = at;
            a.copies[3 * at] = page;
            a.copies[3 * at + 2] = a.P;
        }
    }
    __syncthreads();
    for (int i = tid; i < a.n_copies; i += kPlanThreads) {
        if (i < moves) {
            a.copies[3 * i + 1] = a.list[i];
        } else {
            a.copies[3 * i] = a.copies[3 * i + 1] = -1;
            a.copies[3 * i + 2] = 0;
        }
    }
    if (tid == 0) {
        a.list[-1] = n;
        *a.free_pages = a.n_pages - n;
    }
}

__global__ void __launch_bounds__(256) pages_rename_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int b = (blockIdx.x * 256 + threadIdx.x) / 32, lane = threadIdx.x % 32;
    if (b >= a.n_out) return;
    const Kept k = kept_of(a, b);
    const int n = a.list[-1];
    for (int i = lane; i < a.max_pages; i += 32) {
        int page = -1;
        if (i < k.pages && is_page(a, page = k.old[i])) {
            if (page >= n && !(a.pins[page / 32] >> (page % 32) & 1u)) page = a.list[a.move[page]];
        } else {
            page = -1;
        }
        a.table_out[b * a.out_stride + i] = page;
    }
}

// ------------------------------------------------------------ copies

// Block (c, y): pair c of the list, y = layer * 2 + (0: keys, 1: values).  Vec is what a
// thread moves at once; a row is 2^unit_shift of them, 256 at most.
template <typename Vec>
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagesCopyArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kAhead = 8;
    const int src = a.copies[3 * blockIdx.x], dst = a.copies[3 * blockIdx.x + 1];
    const int rows = min(max(a.copies[3 * blockIdx.x + 2], 0), a.P);
    if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages || src == dst) return;
    // a thread keeps one unit of every few rows of the page's H_kv * rows
    const int units = 1 << a.unit_shift, unit = threadIdx.x & (units - 1), step = 256 >> a.unit_shift;
    const int n = a.H_kv * rows;  // the host has checked that it fits
    for (int y = blockIdx.y; y < 2 * a.layers; y += gridDim.y) {
        const PagesCopyArgs::Side s = y % 2 ? a.v : a.k;
        char *base = s.p + (y / 2) * s.layer + unit * static_cast<long long>(sizeof(Vec));
        const char *from = base + src * s.page;
        char *to = base + dst * s.page;
        for (int i0 = threadIdx.x >> a.unit_shift; i0 < n; i0 += step * kAhead) {
            Vec v[kAhead];
            long long at[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + step * e, h = i / rows;
                at[e] = h * s.head + (i - h * rows) * s.row;
                if (i < n) v[e] = *reinterpret_cast<const Vec *>(from + at[e]);
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (i0 + step * e < n) *reinterpret_cast<Vec *>(to + at[e]) = v[e];
        }
    }
}

cudaError_t launch_clear(const PagesArgs &a) {
    const int blocks = a.words < 8 * 1024 ? (a.words + 7) / 8 : 1024;
    return launch_pdl(pages_clear_kernel, dim3(static_cast<unsigned>(blocks > 0 ? blocks : 1)), dim3(256), 0, a.stream, a);
}

dim3 warps_for(long long rows) { return dim3(static_cast<unsigned>((rows + 7) / 8)); }

}  // namespace

cudaError_t launch_pages_step(const PagesArgs &a) {
    cudaError_t e = launch_clear(a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_mark_kernel, warps_for(a.n_out), dim3(256), 0, a.stream, a);
    if (e == cudaSuccess) e = launch_pdl(pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_write_kernel, warps_for(a.n_out), dim3(256), 0, a.stream, a);
    return e;
}

cudaError_t launch_pages_compact(const PagesArgs &a) {
    cudaError_t e = launch_clear(a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_mark_kernel, warps_for(a.n_out), dim3(256), 0, a.stream, a);
    if (e == cudaSuccess) e = launch_pdl(pages_moves_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_rename_kernel, warps_for(a.n_out), dim3(256), 0, a.stream, a);
    return e;
}

cudaError_t launch_pages_copy(PagesCopyArgs a, bool wide, int esz) {
    a.unit_shift = 0;
    while ((wide ? 16 : esz) << a.unit_shift < a.row_bytes) ++a.unit_shift;
    const dim3 grid(static_cast<unsigned>(a.n_copies), static_cast<unsigned>(2 * a.layers < 65535 ? 2 * a.layers : 65534));
    if (wide) return launch_pdl(pages_copy_kernel<uint4>, grid, dim3(256), 0, a.stream, a);
    return esz == 4 ? launch_pdl(pages_copy_kernel<uint32_t>, grid, dim3(256), 0, a.stream, a)
                    : launch_pdl(pages_copy_kernel<uint16_t>, grid, dim3(256), 0, a.stream, a);
}

}  // namespace attn
