// The table of pages of a paged KV cache, and copies of pages.
//
// attn_pages_step makes the next table from the last one: row b goes on from row
// parents[b], cut back or grown to new_len[b] tokens.  No counts of holders are kept from
// call to call: which pages are held is read off the table, as a set of bits.
//   1. bits = pinned pages
//   2. full pages that stay set their bits; a partly filled page goes to the lowest row
//      that holds it as such
//   3. which rows keep their partly filled page (its first, unless the bit says that
//      another row holds it full or it is pinned), how many new pages each row wants, the
//      prefix sums of both the wants and the free pages of each word of bits, and the list
//      of the lowest free pages, as many as are wanted
//   4. each row is written, and the copy it needs
// Minima, unions and prefix sums do not depend on the order of the threads, so a call gives
// the same table every time.
//
// attn_pages_compact sets the bits of all pages held (n of them) in the same way; the k-th
// lowest held page from n on moves to the k-th lowest free one below n.
//
// Both move a few hundred KB; what bounds them is the chain of dependent steps.  Pools of up
// to 262144 pages, whose bits fit in shared memory, take one launch of a cluster of eight
// CTAs with four barriers (pages_one_kernel): 256 sequences of up to 7000 tokens in pages
// of 16 rows 8.9 us (10 us with a lane's entries of the table read one after the other, 13
// also with a pass over all words for the list, 13.4 as four launches; sixteen CTAs
// change nothing: the chain is the same).  Larger ones take four launches with the bits in
// the workspace: clear, mark (a block a row), plan or moves (one block), write or rename (a
// block a row).  The limits (with 2048 rows) are what shared memory holds, not where the forms
// cross: rows of 512 entries in pools of 262145 and 1048576 pages take the four launches 14.5 and
// 33 us a step, 130 and 565 a compaction (its one block walks all words), and of wide tables eight
// CTAs write less than all SMs do (8192 entries a row, a tenth of them in use and nine tenths;
// step, compaction):
//   256 rows, one launch 26, 55 and 36, 61 us; four launches 18, 121 and 68, 150 us
//   2048 rows, one launch 165, 190 and 240, 373 us; four launches 73, 143 and 261, 328 us
//
// attn_pages_copy moves whole rows of pages, 16 bytes a thread and four in flight, bound by
// HBM: 120 MB read and 120 MB written in 37 us, 6.5 TB/s.  A pair that is none costs its blocks, two
// a layer: some 1 ns each (5 pages of a pool of 100000, whose list has 50000 pairs, 101 us in
// one layer, 3.2 ms in 32).
#include "clusters.cuh"
#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"

#include <climits>

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kNobody = 0x7fffffff;

__device__ __forceinline__ bool is_page(const PagesArgs &a, int page) { return page >= 0 && page < a.n_pages; }

// The kernels behind this one start once all its blocks have passed their wait: what came
// before the call is complete then, and they read the call's inputs before their own wait.
__global__ void __launch_bounds__(256) pages_clear_kernel(const PagesArgs a) {
    griddep_wait();
    griddep_launch_dependents();
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

constexpr int kRowThreads = 128;

// A row's first entries, kEarly of each thread, on their way while the kernel waits.
constexpr int kEarly = 4;
struct Early {
    int page[kEarly];
    __device__ __forceinline__ Early(const int32_t *row, int n) {
#pragma unroll
        for (int y = 0; y < kEarly; ++y) {
            const int i = static_cast<int>(threadIdx.x) + y * kRowThreads;
            page[y] = i < n ? row[i] : -1;
        }
    }
    // take(i, page) for entries [0, n) of the row
    template <typename Take>
    __device__ __forceinline__ void each(const int32_t *row, int n, Take take) const {
#pragma unroll
        for (int y = 0; y < kEarly; ++y) {
            const int i = static_cast<int>(threadIdx.x) + y * kRowThreads;
            if (i < n) take(i, page[y]);
        }
#pragma unroll 4
        for (int i = static_cast<int>(threadIdx.x) + kEarly * kRowThreads; i < n; i += kRowThreads) take(i, row[i]);
    }
};

// One block a row.
__global__ void __launch_bounds__(kRowThreads) pages_mark_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x;
    const Kept k = kept_of(a, b);
    const int whole = a.first ? k.full : k.full + (k.part != 0);  // compaction: every page alike
    const Early early(k.old, whole);
    const int last = k.part ? k.old[k.full] : -1;
    griddep_wait();
    int lost = 0;  // entries that are no pages: asked for anew
    early.each(k.old, whole, [&](int, int page) {
        if (is_page(a, page))
            atomicOr(&a.held[page / 32], 1u << (page % 32));
        else
            ++lost;
    });
    if (!a.first) return;
    if (tid == 0 && is_page(a, last)) atomicMin(&a.first[last], b);
    __shared__ int sums[kRowThreads / 32];
    lost = __reduce_add_sync(0xffffffffu, lost);
    if (tid % 32 == 0) sums[tid / 32] = lost;
    __syncthreads();
    if (tid == 0) {
        int all = 0;
        for (int w = 0; w < kRowThreads / 32; ++w) all += sums[w];
        a.lost[b] = all;
    }
}

// Sum of the values of the threads before this one, and of all of them.  The whole block
// calls it.
__device__ __forceinline__ int block_prefix(unsigned v, int *total) {
    __shared__ unsigned sums[kPlanThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    unsigned s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    unsigned w = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const unsigned before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    __syncthreads();
    return static_cast<int>(s - v + (warp ? before : 0u));
}

__device__ __forceinline__ unsigned pages_of_word(const PagesArgs &a, int w) {  // bits that stand for a page
    const int n = a.n_pages - w * 32;
    return n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Calls take(page, k) for the k-th set bit of the words that the first `n` threads hold (w0 +
// thread, its first bit the at-th, in order), a lane a bit: neighbours write side by side.  k
// from `most` on is left out.  The whole block calls it.
template <typename Take>
__device__ __forceinline__ void each_bit(int w0, int n, unsigned bits, int at, int most, Take take) {
    __shared__ int2 words[kPlanThreads];
    words[threadIdx.x] = make_int2(static_cast<int>(bits), at);
    __syncthreads();
    const int lane = threadIdx.x % 32;
    for (int w = threadIdx.x / 32; w < min(n, kPlanThreads); w += kPlanThreads / 32) {
        const int2 x = words[w];
        const unsigned set = static_cast<unsigned>(x.x);
        if (x.y >= most) break;
        const int k = x.y + __popc(set & ((1u << lane) - 1u));
        if ((set >> lane & 1u) && k < most) take((w0 + w) * 32 + lane, k);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    // rows: who keeps its partly filled page, and the wants
    int wants = 0;
    for (int b0 = 0; b0 == 0 || b0 < a.n_out; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int want = 0, page = -1;
        Kept k{};
        if (b < a.n_out) {
            k = kept_of(a, b);
            if (k.part) page = k.old[k.full];
        }
        if (b0 == 0) griddep_wait();
        if (b < a.n_out) {
            const int lost = a.lost[b];
            int stays = 0;
            if (k.part) {
                // a row whose page this is sets the bit below: no other row is its first
                if (is_page(a, page) && a.first[page] == b && !(*const_cast<volatile unsigned *>(&a.held[page / 32]) >> (page % 32) & 1u)) {
                    stays = 1;
                    atomicOr(&a.held[page / 32], 1u << (page % 32));
                }
            }
            want = lost + k.pages - k.full - stays;
            a.stays[b] = stays;
        }
        int all;
        const int at = wants + block_prefix(want, &all);
        if (b < a.n_out) a.need[b] = at;  // the row's first new page in the list
        wants += all;
    }
    __syncthreads();  // the bits set above
    int free_pages = 0;
    for (int w0 = 0; w0 < a.words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        const unsigned bits = w < a.words ? ~*const_cast<volatile unsigned *>(&a.held[w]) & pages_of_word(a, w) : 0u;
        int all;
        const int at = free_pages + block_prefix(__popc(bits), &all);
        each_bit(w0, a.words - w0, bits, at, wants, [&](int page, int k) { a.list[k] = page; });
        free_pages += all;
    }
    if (tid == 0) {
        a.list[-1] = free_pages;
        *a.free_pages = free_pages - wants;
    }
}

// One block a row.
__global__ void __launch_bounds__(kRowThreads) pages_write_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x;
    const Kept k = kept_of(a, b);
    const Early early(k.old, k.full + (k.part != 0));
    const int from = k.part ? k.old[k.full] : -1;
    griddep_wait();
    const int stays = a.stays[b], n_free = a.list[-1], first = a.need[b], lost = a.lost[b];
    const int kept = k.full + stays;
    int32_t *out = a.table_out + b * a.out_stride;
    auto given = [&](int nth) { return nth < n_free ? a.list[nth] : -1; };
    // new pages: entries that are no pages come first, then those behind the kept ones
    if (lost == 0) early.each(k.old, kept, [&](int i, int page) { out[i] = page; });
#pragma unroll 4
    for (int i = kept + tid; i < a.max_pages; i += kRowThreads) out[i] = i < k.pages ? given(first + lost + i - kept) : -1;
    if (lost > 0 && tid < 32) {  // rare: one warp counts its way through them
        int nth = first;
        for (int i0 = 0; i0 < kept; i0 += 32) {
            const int i = i0 + tid;
            int page = i < kept ? k.old[i] : 0;
            const bool wanted = i < kept && !is_page(a, page);
            const unsigned all = __ballot_sync(0xffffffffu, wanted);
            if (wanted) page = given(nth + __popc(all & ((1u << tid) - 1u)));
            nth += __popc(all);
            if (i < kept) out[i] = page;
        }
    }
    if (tid == kRowThreads - 1) {
        a.len_out[b] = k.len;
        // a page not kept is the first entry behind those that are
        const int to = k.part && !stays ? given(first + lost) : -1;
        const bool copied = is_page(a, from) && to >= 0;
        a.copies[3 * b] = copied ? from : -1;
        a.copies[3 * b + 1] = copied ? to : -1;
        a.copies[3 * b + 2] = copied ? k.part : 0;
    }
}

// Compaction: n pages are held or pinned; the movable ones from n on go to the free ones
// below n.
__global__ void __launch_bounds__(kPlanThreads) pages_moves_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x;
    int n = 0;
    for (int w = tid; w < a.words; w += kPlanThreads) n += __popc(a.held[w]);
    int all;
    block_prefix(n, &all);
    n = all;
    auto below = [&](int w) { return n - w * 32 >= 32 ? 0xffffffffu : n > w * 32 ? (1u << (n - w * 32)) - 1u : 0u; };  // pages < n
    int holes = 0, moves = 0;
    for (int w0 = 0; w0 * 32 < n; w0 += kPlanThreads) {
        const int w = w0 + tid;
        const unsigned bits = w < a.words ? ~a.held[w] & below(w) : 0u;
        const int at = holes + block_prefix(__popc(bits), &all);
        each_bit(w0, a.words - w0, bits, at, INT_MAX, [&](int page, int k) { a.list[k] = page; });
        holes += all;
    }
    for (int w0 = n / 32 / kPlanThreads * kPlanThreads; w0 < a.words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        const unsigned bits = w < a.words ? a.held[w] & ~below(w) & ~a.pins[w] : 0u;
        const int at = moves + block_prefix(__popc(bits), &all);
        each_bit(w0, a.words - w0, bits, at, INT_MAX, [&](int page, int k) {
            const int to = a.list[k];
            a.move[page] = to;
            a.copies[3 * k] = page;
            a.copies[3 * k + 1] = to;
            a.copies[3 * k + 2] = a.P;
        });
        moves += all;
    }
    for (int i = moves + tid; i < a.n_copies; i += kPlanThreads) {
        a.copies[3 * i] = a.copies[3 * i + 1] = -1;
        a.copies[3 * i + 2] = 0;
    }
    if (tid == 0) {
        a.list[-1] = n;
        *a.free_pages = a.n_pages - n;
    }
}

// One block a row.
__global__ void __launch_bounds__(kRowThreads) pages_rename_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    const int b = blockIdx.x;
    const Kept k = kept_of(a, b);
    const Early early(k.old, k.pages);
    griddep_wait();
    const int n = a.list[-1];
    int32_t *out = a.table_out + b * a.out_stride;
    early.each(k.old, k.pages, [&](int i, int page) {
        if (is_page(a, page)) {
            const int to = a.move[page];  // of a page that moves
            if (page >= n && !(a.pins[page / 32] >> (page % 32) & 1u)) page = to;
        } else {
            page = -1;
        }
        out[i] = page;
    });
    for (int i = k.pages + static_cast<int>(threadIdx.x); i < a.max_pages; i += kRowThreads) out[i] = -1;
}

// ------------------------------------------------------------ both in one launch

// Pools of up to kOneMaxPages and tables of up to kOneMaxRows: one cluster of eight CTAs goes
// through the same steps, with the bits in shared memory.  A CTA marks the pages of every
// eighth row in bits of its own, then owns an eighth of the words, of all CTAs together.
constexpr int kOne = 8;
constexpr int kOneMaxPages = 1 << 18, kOneMaxRows = 2048;
constexpr int kOneWords = kOneMaxPages / 32;
struct OneSmem {
    unsigned marks[kOneWords];                // of this CTA's rows
    unsigned held[kOneWords / kOne], pins[kOneWords / kOne];  // this CTA's words
    unsigned used[kOneWords / kOne];          // step: held, or some row's partly filled page
    int last[kOneMaxRows];                    // a row's partly filled page or -1 (every CTA has them all)
    int want[kOneMaxRows];                    // new pages a row wants, then its first in the list
    Kept kept[kOneMaxRows / kOne];            // of this CTA's rows
    int lost[kOneMaxRows / kOne], stays[kOneMaxRows / kOne];
    unsigned total[kOne];                     // step: free pages of each CTA's words; compaction: pages held
                                              // and, 16 bits up, those that may move
    int most;                                 // step: new pages that the rows want at most
};
static_assert(kOneWords / kOne == kPlanThreads, "a thread a word");

__device__ __forceinline__ void store_remote(const void *p, unsigned rank, int v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_rank(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned load_remote(const void *p, unsigned rank) {
    unsigned v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_rank(p, rank)) : "memory");
    return v;
}

template <bool Step>
__global__ void __launch_bounds__(kPlanThreads, 1) pages_one_kernel(const PagesArgs a) {
    extern __shared__ __align__(16) uint8_t one_smem[];
    OneSmem &sm = *reinterpret_cast<OneSmem *>(one_smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const unsigned rank = cluster_rank();
    const int each = max(1, (a.words + kOne - 1) / kOne);  // words of a CTA
    const int w = static_cast<int>(rank) * each + tid;     // this thread's word
    const bool mine = tid < each && w < a.words;
    constexpr int kStride = kOne * (kPlanThreads / 32);    // rows of a pass
    constexpr int kBatch = 16;                             // entries on their way to a lane
    const int row0 = static_cast<int>(rank) + kOne * warp;
    for (int i = tid; i < a.words; i += kPlanThreads) sm.marks[i] = 0;
    if (tid == 0) sm.most = 0;
    cluster_sync();  // every CTA runs: its shared memory may be written
    griddep_launch_dependents();
    griddep_wait();
    // ---- marks of this CTA's rows
    for (int b = row0; b < a.n_out; b += kStride) {
        const Kept k = kept_of(a, b);
        const int whole = Step ? k.full : k.full + (k.part != 0);
        int32_t *out = a.table_out + b * a.out_stride;
        int lost = 0, last = Step && k.part ? k.old[k.full] : -1;
        for (int i0 = lane; i0 < whole; i0 += 32 * kBatch) {
            int page[kBatch];
#pragma unroll
            for (int y = 0; y < kBatch; ++y) page[y] = i0 + 32 * y < whole ? k.old[i0 + 32 * y] : -1;
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                if (i0 + 32 * y >= whole) break;
                if (is_page(a, page[y]))
                    atomicOr(&sm.marks[page[y] / 32], 1u << (page[y] % 32));
                else
                    ++lost;
                if (Step) out[i0 + 32 * y] = page[y];  // those that are no pages get others below
            }
        }
        if (Step) {
#pragma unroll 4
            for (int i = k.pages + lane; i < a.max_pages; i += 32) out[i] = -1;
            lost = __reduce_add_sync(0xffffffffu, lost);
            if (!is_page(a, last)) last = -1;
            if (lane < kOne) {
                store_remote(&sm.last[b], static_cast<unsigned>(lane), last);
                asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(map_rank(&sm.most, static_cast<unsigned>(lane))),
                             "r"(lost + k.pages - k.full) : "memory");
            }
            if (lane == 0) sm.lost[b / kOne] = lost;
        }
        if (lane == 0) sm.kept[b / kOne] = k;
    }
    // ---- pinned pages of this CTA's words, a lane a page
    if (a.pinned) {
        for (int i = warp; i < each; i += kPlanThreads / 32) {
            const int page = (static_cast<int>(rank) * each + i) * 32 + lane;
            const unsigned bits = __ballot_sync(0xffffffffu, page < a.n_pages && a.pinned[page] != 0);
            if (lane == 0) sm.pins[i] = bits;
        }
    } else if (tid < each) {
        sm.pins[tid] = 0;
    }
    cluster_sync();
    // ---- this CTA's words, of all rows
    const int w0 = static_cast<int>(rank) * each;
    unsigned held = 0, pins = 0;
    if (mine) {
        held = pins = sm.pins[tid];
#pragma unroll
        for (unsigned y = 0; y < kOne; ++y) held |= load_remote(&sm.marks[w], y);
        sm.held[tid] = held;
    }
    int wants = 0, given_out = 0;  // step: new pages wanted, and there to be given out
    int n = 0, moves = 0;          // compaction: pages held, pages that move
    if (Step) {
        // A partly filled page of any row is not free, whoever keeps it: full, pinned or this.
        if (mine) sm.used[tid] = held;
        __syncthreads();
        for (int b = tid; b < a.n_out; b += kPlanThreads) {
            const int page = sm.last[b], at = page / 32 - w0;
            if (page >= 0 && at >= 0 && at < each) atomicOr(&sm.used[at], 1u << (page % 32));
        }
        __syncthreads();
        const unsigned free_bits = mine ? ~sm.used[tid] & pages_of_word(a, w) : 0u;
        int all;
        int at = block_prefix(__popc(free_bits), &all);
        if (tid < kOne) store_remote(&sm.total[rank], static_cast<unsigned>(tid), all);
        cluster_sync();
        // ---- which rows keep their partly filled page, and what each wants
        for (int b = row0; b < a.n_out; b += kStride) {
            const Kept k = sm.kept[b / kOne];
            const int page = sm.last[b];
            int stays = 0;
            if (page >= 0) {
                const unsigned bits = load_remote(&sm.held[page / 32 % each], static_cast<unsigned>(page / 32 / each));
                bool first = true;
                for (int y = lane; y < b; y += 32) first = first && sm.last[y] != page;
                stays = __all_sync(0xffffffffu, first) && !(bits >> (page % 32) & 1u);
            }
            const int lost = sm.lost[b / kOne];
            if (lane < kOne) store_remote(&sm.want[b], static_cast<unsigned>(lane), lost + k.pages - k.full - stays);
            if (lane == 0) sm.stays[b / kOne] = stays;
        }
        // ---- the list of free pages, as far as they may be wanted
        for (int y = 0; y < kOne; ++y) {
            if (y == static_cast<int>(rank)) at += given_out;
            given_out += static_cast<int>(sm.total[y]);
        }
        each_bit(w0, each, free_bits, at, sm.most, [&](int page, int k) { a.list[k] = page; });
        __threadfence();
        cluster_sync();
        // ---- the places of the rows' wants in it
        for (int b0 = 0; b0 < a.n_out; b0 += kPlanThreads) {
            const int b = b0 + tid;
            const int first = wants + block_prefix(b < a.n_out ? sm.want[b] : 0, &all);
            if (b < a.n_out) sm.want[b] = first;
            wants += all;
        }
        __syncthreads();
    } else {
        int all;
        const unsigned movable = held & ~pins;
        const unsigned before = block_prefix(__popc(held) | static_cast<unsigned>(__popc(movable)) << 16, &all);  // at most 2^15 each
        if (tid < kOne) store_remote(&sm.total[rank], static_cast<unsigned>(tid), all);
        cluster_sync();
        // held pages before this word, those of them that may move, and of the latter those below page n
        int held_at = static_cast<int>(before & 0xffffu), movable_at = static_cast<int>(before >> 16), below_n = 0;
        for (int y = 0; y < kOne; ++y) {
            if (y == static_cast<int>(rank)) held_at += n, movable_at += moves;
            n += static_cast<int>(sm.total[y] & 0xffffu);
            moves += static_cast<int>(sm.total[y] >> 16);
        }
        const int owner = n / 32 / each;  // of page n
        for (int y = 0; y < owner && y < kOne; ++y) below_n += static_cast<int>(sm.total[y] >> 16);
        auto below = [&](int x) { return n - x * 32 >= 32 ? 0xffffffffu : n > x * 32 ? (1u << (n - x * 32)) - 1u : 0u; };  // pages < n
        const int word = owner * each + tid;
        int part = 0;
        if (tid < each && word * 32 < n) {
            const unsigned there = static_cast<unsigned>(owner);
            part = __popc(load_remote(&sm.held[tid], there) & ~load_remote(&sm.pins[tid], there) & below(word));
        }
        block_prefix(part, &all);
        below_n += all;
        moves -= below_n;
        // the free pages before a word are those that are not held
        each_bit(w0, each, mine ? ~held & below(w) : 0u, w * 32 - held_at, INT_MAX, [&](int page, int k) { a.list[k] = page; });
        each_bit(w0, each, movable & ~below(w), movable_at + __popc(movable & below(w)) - below_n, INT_MAX, [&](int page, int k) {
            a.move[page] = k;
            a.copies[3 * k] = page;
            a.copies[3 * k + 2] = a.P;
        });
        if (a.pinned) each_bit(w0, each, held & ~below(w) & pins, 0, INT_MAX, [&](int page, int) { a.move[page] = -1; });
        __threadfence();
        cluster_sync();
    }
    // ---- the new rows
    if (rank == 0 && tid == 0) *a.free_pages = Step ? given_out - wants : a.n_pages - n;
    for (int b = row0; b < a.n_out; b += kStride) {
        const Kept k = sm.kept[b / kOne];
        int32_t *out = a.table_out + b * a.out_stride;
        if (!Step) {
            for (int i0 = lane; i0 < a.max_pages; i0 += 32 * kBatch) {
                int page[kBatch];
#pragma unroll
                for (int y = 0; y < kBatch; ++y) page[y] = i0 + 32 * y < k.pages ? k.old[i0 + 32 * y] : -1;
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    if (!is_page(a, page[y])) page[y] = -1;
                    const int to = page[y] >= n ? __ldcg(&a.move[page[y]]) : -1;
                    if (to >= 0) page[y] = __ldcg(&a.list[to]);
                }
#pragma unroll
                for (int y = 0; y < kBatch; ++y)
                    if (i0 + 32 * y < a.max_pages) out[i0 + 32 * y] = page[y];
            }
            continue;
        }
        const int stays = sm.stays[b / kOne], lost = sm.lost[b / kOne], first = sm.want[b], kept = k.full + stays;
        auto given = [&](int nth) { return nth < given_out ? __ldcg(&a.list[nth]) : -1; };
        if (stays && lane == 0) out[k.full] = sm.last[b];
#pragma unroll 4
        for (int i = kept + lane; i < k.pages; i += 32) out[i] = given(first + lost + i - kept);
        if (lost > 0) {  // rare: entries that are no pages get the first of the new ones
            int nth = first;
            for (int i0 = 0; i0 < k.full; i0 += 32) {
                const int i = i0 + lane;
                const bool wanted = i < k.full && !is_page(a, k.old[i]);
                const unsigned some = __ballot_sync(0xffffffffu, wanted);
                if (wanted) out[i] = given(nth + __popc(some & ((1u << lane) - 1u)));
                nth += __popc(some);
            }
        }
        if (lane == 0) {
            a.len_out[b] = k.len;
            const int source = sm.last[b], to = k.part && !stays ? given(first + lost) : -1;
            const bool copied = source >= 0 && to >= 0;
            a.copies[3 * b] = copied ? source : -1;
            a.copies[3 * b + 1] = copied ? to : -1;
            a.copies[3 * b + 2] = copied ? k.part : 0;
        }
    }
    if (!Step)
        for (int i = static_cast<int>(rank) * kPlanThreads + tid; i < a.n_copies; i += kOne * kPlanThreads) {
            if (i < moves) {
                a.copies[3 * i + 1] = __ldcg(&a.list[i]);
            } else {
                a.copies[3 * i] = a.copies[3 * i + 1] = -1;
                a.copies[3 * i + 2] = 0;
            }
        }
}

template <bool Step>
cudaError_t launch_one(const PagesArgs &a) {
    cudaError_t e = cudaFuncSetAttribute(pages_one_kernel<Step>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(OneSmem));
    if (e != cudaSuccess) return e;
    return launch_clusters(pages_one_kernel<Step>, kOne, kOne, kPlanThreads, sizeof(OneSmem), a.stream, a);
}
bool fits_one(const PagesArgs &a) {
    return a.n_pages <= kOneMaxPages && a.n_out <= kOneMaxRows;
}

// ------------------------------------------------------------ copies

// Block (c, y): pair c of the list, y = layer * 2 + (0: keys, 1: values).  Vec is what a
// thread moves at once; a row is 2^unit_shift of them, 256 at most.
template <typename Vec>
__global__ void __launch_bounds__(256, 5) pages_copy_kernel(const PagesCopyArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kAhead = 4;
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

}  // namespace

cudaError_t launch_pages_step(const PagesArgs &a) {
    if (fits_one(a)) return launch_one<true>(a);
    cudaError_t e = launch_clear(a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_mark_kernel, dim3(static_cast<unsigned>(a.n_out)), dim3(kRowThreads), 0, a.stream, a);
    if (e == cudaSuccess) e = launch_pdl(pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_write_kernel, dim3(static_cast<unsigned>(a.n_out)), dim3(kRowThreads), 0, a.stream, a);
    return e;
}

cudaError_t launch_pages_compact(const PagesArgs &a) {
    if (fits_one(a)) return launch_one<false>(a);
    cudaError_t e = launch_clear(a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_mark_kernel, dim3(static_cast<unsigned>(a.n_out)), dim3(kRowThreads), 0, a.stream, a);
    if (e == cudaSuccess) e = launch_pdl(pages_moves_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a);
    if (e == cudaSuccess && a.n_out > 0) e = launch_pdl(pages_rename_kernel, dim3(static_cast<unsigned>(a.n_out)), dim3(kRowThreads), 0, a.stream, a);
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
