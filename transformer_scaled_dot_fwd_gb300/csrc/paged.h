// Internal declarations of the paged KV cache: attention over pages, norm and rotary
// positions with the append to pages, the table of pages.
#pragma once

#include "kernels.h"

namespace attn {

// New tokens over a paged KV cache (attn_fwd_paged).  Sequence s is tokens [cu_seqlens[s],
// cu_seqlens[s + 1]) of q and out, the last of its cache_len[s] keys, which lie in pages
// of P rows named by row s of the page table.
struct PagedArgs {
    const void *q;              // (T, H, D) rows, element strides below
    const void *k, *v;          // pages: (n_pages, H_kv, P, D), element strides below
    void *out;                  // (T, H, D) rows
    float *lse;                 // (T, H) or nullptr
    const int32_t *page_table;  // device, rows table_stride apart
    const int32_t *cu_seqlens;  // device int32[n_seq + 1], or nullptr: per_seq tokens each
    const int32_t *cache_len;   // device int32[n_seq], or nullptr (max_len)
    long long q_ts, q_hs, o_ts, o_hs, k_ps, k_hs, k_rs, v_ps, v_hs, v_rs, table_stride;
    int T, n_seq, per_seq, H, H_kv, D, P, n_pages;
    int max_len;                // keys that a row of the page table holds
    unsigned page_magic;        // ceil(2^32 / P) where that divides every key exactly, or 0
    float scale;
    // bf16: row tiles of `tokens` tokens by `heads` heads of one of `groups` groups of
    // the query heads of a cached head; boxes of `box` rows of a page, box_tokens tokens of q
    int heads, groups, tokens, box, box_tokens;
    // the pages' views: head h of page p is entry p pstep + h hstep; halves: boxes of 64 columns
    int halves, k_pstep, k_hstep, v_pstep, v_hstep;
    int single;                 // every unit has one row tile
    int cluster;                // > 0: every unit is a cluster of so many CTAs, 1 << cluster_shift; no workspace
    int cluster_shift;
    int grid;                   // CTAs at most
    int n_split;                // fp32: splits of the keys
    // Partial results: O unnormalised [D] and (running max in log2 units, sum) of
    // bf16: two slots per CTA of slot_rows rows, O as [slot][D / 4][row][4]
    // fp32: row (((block of 32 rows) * H_kv + cached head) * 32 + r) * n_split + split
    float *part_o, *part_ml;
    int slot_rows;
    int *merge;                 // bf16: 8 ints per CTA, the unit it shares with later CTAs
    int *status;
    cudaStream_t stream;
    int n_sm;
};
// bf16 tcgen05 kernel and its merge; tq views q as (D, H, T) with 64 x heads x box_tokens
// boxes, tk and tv the pages as (64, 8, D / 64, P / 8, heads of pages) with 64 x 8 x D / 64 x
// box / 8 x 1 boxes (halves: as (D, P, H_kv, n_pages) with 64 x 8 x 1 x 1 boxes).
cudaError_t launch_paged_tc(const PagedArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv);
double paged_tc_axis(const PagedArgs &a);
constexpr int kPagedCluster = 8;  // CTAs of a cluster at most
cudaError_t launch_paged_f32(const PagedArgs &a);
// fp32: blocks of 32 rows of a cached head, and splits of the keys (1, 2, 4 or 8: CTAs of
// a cluster; more: merged through the workspace).
long long paged_f32_blocks(const PagedArgs &a);
int paged_f32_splits(const PagedArgs &a);

__device__ __forceinline__ bool is_page(const PagedArgs &a, int page) { return page >= 0 && page < a.n_pages; }
// Entry of the page table that holds a key (a division is some 40 instructions).
__device__ __forceinline__ int page_of_key(const PagedArgs &a, int key) {
    return a.page_magic ? static_cast<int>(__umulhi(static_cast<unsigned>(key), a.page_magic)) : key / a.P;
}

// RMS norm of head rows, rotary positions, and their append to pages (attn_norm_rope,
// attn_rope_append_paged).  Rows are (token, head) with element strides.
struct NormRopeArgs {
    const void *q, *k, *v;      // (T, H | H_kv, D); v only to append
    void *q_out, *k_out;        // k_out may be nullptr to append
    const void *q_weight, *k_weight;  // (D,) or nullptr: the tensor is turned as it is
    void *kpages, *vpages;      // (n_pages, H_kv, P, D), element strides below
    const int32_t *page_table;  // device, rows table_stride apart
    const int32_t *cu_seqlens;  // device int32[n_seq + 1] or nullptr (T / n_seq tokens each)
    const int32_t *cache_len;   // device int32[n_seq] or nullptr (max_len)
    const int32_t *positions;   // device int32[T] or nullptr (the cache row)
    long long q_ts, q_hs, k_ts, kt_hs, v_ts, vt_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    long long k_ps, k_hs, k_rs, v_ps, v_hs, v_rs, table_stride;
    int T, H, H_kv, D, n_seq, P, n_pages, max_len;
    int append;                 // 0: no cache
    int rotary_dim, interleaved;
    float mscale, eps;
    int n_sm;
    cudaStream_t stream;
    uint64_t turns[64];         // w_p / 2 pi as a fraction of 2^64
};
// wide: every address, stride and pair allows 16-byte accesses
cudaError_t launch_norm_rope(const NormRopeArgs &a, bool f32, bool wide);

// The table of pages (attn_pages_step, attn_pages_compact).
struct PagesArgs {
    const int32_t *table;       // (n_seq, max_pages), rows table_stride apart
    const int32_t *cache_len;   // (n_seq) or nullptr (rows full)
    const int32_t *parents;     // (n_out) or nullptr (row b goes on from row b)
    const int32_t *new_len;     // (n_out) or nullptr (the parent's length)
    const int32_t *pinned;      // (n_pages), not 0: held elsewhere too; or nullptr
    int32_t *table_out;         // (n_out, max_pages), rows out_stride apart
    int32_t *len_out;           // (n_out); step only
    int32_t *copies;            // (n_copies, 3): from, to, rows
    int32_t *free_pages;        // (1)
    long long table_stride, out_stride;
    int n_seq, n_out, max_pages, P, n_pages, n_copies;
    // workspace
    int words;                  // of 32 pages
    unsigned *held, *pins;      // bits
    int32_t *first;             // step: (n_pages), the lowest row that holds a page partly filled
    int32_t *need, *stays, *lost;  // step: (n_out)
    int32_t *list;              // pages to be given out (list[-1]: their number, or that of the pages held)
    int32_t *move;              // compact: (n_pages), a moved page's place in the list
    cudaStream_t stream;
};
cudaError_t launch_pages_step(const PagesArgs &a);
cudaError_t launch_pages_compact(const PagesArgs &a);

// Copies of pages (attn_pages_copy).  Strides in bytes.
struct PagesCopyArgs {
    struct Side {
        char *p;
        long long layer, page, head, row;
    } k, v;
    const int32_t *copies;      // (n_copies, 3)
    int n_copies, layers, n_pages, H_kv, P, row_bytes, unit_shift;
    cudaStream_t stream;
};
// wide: every address and stride allows 16-byte accesses
cudaError_t launch_pages_copy(PagesCopyArgs a, bool wide, int esz);

}  // namespace attn
