// Internal interface between the C-ABI shim (api.cu) and the kernel files.
// Arguments arrive here already validated by the shim.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// Launch with programmatic stream serialisation: the kernel may be placed
// while the previous kernel in the stream finishes, and waits for it
// (griddepcontrol.wait) before it reads its inputs or writes anything, so
// back-to-back launches do not pay the full launch gap.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

struct FwdArgs {
    const void *q, *k, *v;  // (B, H, Sq|Skv, D), device
    void *out;              // (B, H, Sq, D), device
    const int32_t *kv_len;  // device int32[B] or nullptr
    int B, H, Sq, Skv, D;
    float scale;            // multiplier of Q K^T
    int causal;
    int *status;            // device status word
    cudaStream_t stream;
    int n_sm;               // streaming multiprocessors on the device
    int H_kv;               // key/value heads (divides H); query head h reads head h / (H / H_kv)
    // Chunk-against-cache mode (attn_fwd_chunked): kv_len[b] is the cached
    // length L_b, query i sits at position L_b - Sq + i (causal), and no query
    // row is treated as padding.
    int chunked;
    float *lse;             // (B, H, Sq) natural-log log-sum-exp of each row, or nullptr
};

// Packed sequences (attn_fwd_packed): FwdArgs with B = number of sequences and
// Sq = Skv = T rows of all sequences together; kv_len is nullptr.
struct PackedArgs : FwdArgs {
    const int32_t *cu_seqlens;  // device int32[B + 1]
    const int4 *plan;           // device: PackedPlan header, then its tile list
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;  // element strides of a token, of a head
};

// What the plan kernel of a bf16 packed call writes to the caller's workspace:
// one header entry and one int4 {first token, length, tile, -} per query-tile
// unit of any head, longest rows first.
struct PackedPlan {
    int n_tiles, group, front, n_items;
};
// Rows of a tile unit: query-tile pairs, or single tiles when heads are paired.
inline int packed_unit_rows(int H, int H_kv) { return ((H / H_kv) & 1) == 0 ? 128 : 256; }
inline long long packed_plan_tiles(long long T, long long n_seq, int unit_rows) { return T / unit_rows + n_seq; }

// bf16 tcgen05 packed prefill: plan kernel, then the prefill kernel.  tq/tk/tv
// view (D, T, heads) with 64 x 128 x 1 boxes; plan_tiles entries follow the header.
cudaError_t launch_packed_tc(const PackedArgs &a, long long plan_tiles, const CUtensorMap &tq, const CUtensorMap &tk,
                             const CUtensorMap &tv);
// fp32 packed prefill on the CUDA cores (no workspace).
cudaError_t launch_packed_f32(const PackedArgs &a);
long long packed_f32_blocks(long long T, long long n_seq);  // of one head

// A tree of T drafted tokens per sequence against a KV cache (attn_decode_tree).
// Row r of key/value head g is query head g * G + r / T, token r % T.
constexpr int kTreeMaxTokens = 128;
struct TreeArgs {
    const void *q;              // (B, H, T, D) rows, element strides below
    const void *k, *v;          // (B, H_kv, Skv, D)
    void *out;                  // (B, H, T, D) rows
    const int32_t *parents;     // device int32, parents_bs apart per sequence (0: one tree for all)
    const int32_t *cache_len;   // device int32[B] or nullptr (Skv)
    const int32_t *draft_len;   // device int32[B] or nullptr (T)
    long long parents_bs, q_bs, q_hs, q_ts, o_bs, o_hs, o_ts;
    int B, H, H_kv, T, Skv, D;
    float scale;
    int chunk, n_split;         // fp32: keys per split and splits; bf16: n_split CTAs
    // Partial results: O unnormalised [D] and (running max in log2 units, sum) of
    // fp32: row ((b * H_kv + g) * G * T + r) * n_split + split
    // bf16: two slots per CTA of slot_rows rows, O as [slot][D / 4][row][4] (tree_tc.cu)
    float *part_o, *part_ml;
    int *merge;                 // bf16: 8 ints per CTA, the unit it shares with later CTAs
    int *status;
    cudaStream_t stream;
    int n_sm;
};
// fp32: keys per split for these sizes.  Splits of up to kTreeClusterF32 (a power of two
// of them) are the CTAs of a cluster and need no workspace.
constexpr int kTreeClusterF32 = 8;
inline int tree_splits_f32(int Skv, int chunk) {
    const int n = (Skv + chunk - 1) / chunk;
    return n <= 2 || n > kTreeClusterF32 ? n : n <= 4 ? 4 : 8;
}
int tree_chunk_f32(int B, int H, int H_kv, int T, int Skv, int D, int n_sm);
// bf16: CTAs for these sizes (-1: too large), and rows of a workspace slot.
int tree_tc_grid(int B, int H, int H_kv, int T, int Skv, int n_sm);
int tree_tc_slot_rows(int H, int H_kv, int T);
// bf16 tcgen05 kernel and its merge; tk/tv view the caches as (D, Skv, B * H_kv) with 64 x 128 x 1 boxes.
cudaError_t launch_tree_tc(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv);
cudaError_t launch_tree_zero(const TreeArgs &a);  // bf16, Skv = 0
cudaError_t launch_tree_f32(const TreeArgs &a);
cudaError_t launch_tree_merge_f32(const TreeArgs &a);

struct DecodeArgs {
    const void *q;          // (B, H, D) bf16 (fp32 for launch_decode_f32)
    const void *k, *v;      // (B, H_kv, Skv, D), same dtype
    void *out;              // (B, H, D), same dtype
    const int32_t *kv_len;  // device int32[B] or nullptr
    int B, H, Skv, D;
    float scale;
    int chunk;              // keys per split (multiple of 64, <= kDecodeMaxChunk)
    int n_split;            // ceil(Skv / chunk), >= 1
    float *part_o;          // B*H*n_split*D fp32 partial outputs
    float *part_ml;         // B*H*n_split*2 fp32 (running max in log2 units, sum)
    int *status;
    cudaStream_t stream;
    int H_kv;               // cached heads (divides H); query head h reads head h / (H / H_kv)
};

constexpr int kDecodeMaxChunk = 1024;
constexpr int kDecodeGqaMaxChunk = 512;

// Debug attention (attn_fwd_debug): any d_k, d_v <= 256, optional weights.
struct DebugArgs {
    const void *q, *k, *v;  // (B, H, Sq, Dk), (B, H_kv, Skv, Dk), (B, H_kv, Skv, Dv)
    void *out;              // (B, H, Sq, Dv), input dtype
    float *weights;         // (B, H, Sq, Skv) fp32 or nullptr
    const int32_t *kv_len;  // device int32[B] or nullptr
    int B, H, H_kv, Sq, Skv, Dk, Dv;
    float scale;
    int causal;
    int dtype_bf16;
    cudaStream_t stream;
};
cudaError_t launch_debug_attention(const DebugArgs &a);

// fp32 SIMT prefill (D in {64, 128}).
cudaError_t launch_prefill_f32(const FwdArgs &a);

// bf16 tcgen05 prefill (D in {64, 128}); tq/tk/tv are 3-D tensor maps over
// (D, S, B*H) with 64 x 128 x 1 boxes and 128-byte swizzle.
cudaError_t launch_prefill_tc(const FwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv);

// Clears every work counter of the bf16 prefill kernels on the current device
// (synchronous; no prefill launch may be in flight).
cudaError_t reset_prefill_counters();

// bf16 split-KV decode: partial kernel then combine kernel.
cudaError_t launch_decode(const DecodeArgs &a);

// The combine kernel alone (per query head: merge the chunk partials).
cudaError_t launch_decode_combine(const DecodeArgs &a);

// Grouped-query decode (H_kv < H): partial kernel per (b, h_kv, head subgroup,
// chunk), then the combine kernel.  a.chunk must not exceed
// kDecodeGqaMaxChunk (the kernel's score buffer holds that many keys).
cudaError_t launch_decode_gqa(const DecodeArgs &a);
int decode_gqa_heads_per_cta(int G);

// fp32 decode (any grouping H_kv | H): q, caches and out are fp32; partial
// kernel per (b, h, chunk <= kDecodeMaxChunk keys) on the CUDA cores, then an
// fp32-output combine.
cudaError_t launch_decode_f32(const DecodeArgs &a);

// Grouped-query / multi-query decode on the tensor cores (G = H / H_kv query
// heads per cached head, kDecodeTcMinGroup <= G <= 128; below that the CUDA-core
// kernels are as fast or faster): the G queries are the
// rows of one 128-row tile.  tq views q as (D, B*H) with 64 x 128 boxes; tk, tv
// view the caches as (D, Skv, B*H_kv) with 64 x 64 x 1 boxes (128-byte swizzle).
// a.chunk (a multiple of 64 keys, from decode_tc_chunk) and a.n_split as for
// the other decode kernels; the partials are merged by the decode combine.
#ifndef ATTN_DTC_MIN_GROUP
#define ATTN_DTC_MIN_GROUP 4
#endif
constexpr int kDecodeTcMinGroup = ATTN_DTC_MIN_GROUP;
int decode_tc_chunk(int B, int H_kv, int Skv, int n_sm);
cudaError_t launch_decode_tc(const DecodeArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                             const CUtensorMap &tv);

// Rotary positions (attn_rope, attn_rope_append).  Rows are (token, head) with
// element strides.
constexpr int kRopeMaxTokens = 2;  // tokens a block takes at most
struct RopeArgs {
    const void *q, *k, *v;      // (T, H | H_kv, D); v only to append
    void *q_out, *k_out;        // k_out may be nullptr to append
    void *kcache, *vcache;      // (B, H_kv, Skv, D); nullptr without rows
    const int32_t *cu_seqlens;  // device int32[B + 1] or nullptr (T / B tokens each)
    const int32_t *cache_len;   // device int32[B] or nullptr (Skv)
    const int32_t *positions;   // device int32[T] or nullptr (the cache row)
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    int T, H, H_kv, D, B, Skv;
    int append;                 // 0: no cache (Skv = 0 is a cache of no rows)
    int rotary_dim, interleaved;
    float mscale, sin_scale;    // multipliers of cos and of sin (negative sin_scale: inverse)
    int n_sm;
    cudaStream_t stream;
    uint64_t turns[64];         // w_p / 2 pi as a fraction of 2^64
};
// wide: every address, stride and rotary_dim / 2 allows 16-byte accesses
cudaError_t launch_rope(const RopeArgs &a, bool f32, bool wide);

// Size of the library-static decode scratch used by attn_decode_noalloc.
constexpr size_t kDecodeNoAllocScratchBytes = 32u << 20;

// Decode with its partials in the library-static scratch (no allocation).
// The caller has checked that the partials fit in kDecodeNoAllocScratchBytes.
cudaError_t launch_decode_noalloc(DecodeArgs a, bool f32);

// One-warp kernel whose only wait can never complete: exercises the bounded
// wait and the status word (attn_selftest_wait_timeout).
cudaError_t launch_wait_timeout_probe(long long limit, int *status, cudaStream_t stream);

// Writes zeros over n bytes (multiple of 16, 16-byte aligned) -- degenerate
// calls whose every row sees no key.
cudaError_t launch_zero_fill(void *out, size_t n_bytes, cudaStream_t stream);

}  // namespace attn
