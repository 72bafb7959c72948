/*
 * attn.h -- C ABI of the GB300 (sm_103a) scaled dot-product attention library.
 *
 * The library computes multi-head scaled dot-product attention forward,
 *
 *     out = softmax(Q K^T * scale + M) V        independently per (batch, head),
 *
 * where M is 0 for an allowed (query, key) pair and -inf for a forbidden one,
 * applied before the softmax.  The definition is the one shared by the pages
 * "Attention from First Principles" (section 1, "In one line"; section 4,
 * "Tiny example"), "Self-Attention" ("Scaled Dot-Product Attention", "Causal
 * Masking") and "Attention from Scratch" (kube-dojo), Parts 2 and 3.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout.   Tensors are dense, row-major (B, H, S, D) arrays with D fastest:
 *           element (b, h, s, d) lives at ((b*H + h)*S + s)*D + d.  This is
 *           the head-split layout of "Attention from scratch"
 *           (open-llm-engineering), split_heads.  Decode tensors q and out are
 *           (B, H, D), i.e. (B, H, 1, D).
 * Memory.   Every tensor pointer is DEVICE memory owned by the caller, aligned
 *           to 16 bytes (a pointer to an empty tensor may be NULL).  The
 *           library never frees or retains it.  kv_len, when
 *           not NULL, is a DEVICE array of B int32 values; it is read by the
 *           kernels (no host synchronisation), and each value is clamped to
 *           [0, Skv].
 * Streams.  `stream` is a cudaStream_t (NULL = the legacy default stream).
 *           Calls are asynchronous: they enqueue work and return.  Argument
 *           errors are detected on the host before anything is enqueued.
 *           Kernels are launched with programmatic stream serialisation
 *           (programmatic dependent launch): one may be placed while the
 *           previous kernel in the stream finishes, but it reads no input
 *           and writes nothing before that kernel has completed, so stream
 *           order holds as for an ordinary launch.
 * dtype.    ATTN_BF16: bfloat16 inputs and output, fp32 accumulation and
 *           softmax statistics, output rounded to nearest even.  On the tensor
 *           cores (every bf16 prefill, attn_decode_tree, attn_fwd_paged, attn_decode_gqa
 *           with 4 to 128 query heads a cached head) the softmax weights are rounded to
 *           bf16 before they multiply V, by at most 2^-8 of each; their sum is
 *           that of the fp32 weights.
 *           ATTN_F32: float32 everywhere (no TF32).  Output dtype = input dtype.
 * Masking.  causal: key j is visible from query i iff j <= i + (Skv - Sq)
 *           (the last query is aligned with the last key; for Sq == Skv this
 *           is the lower-triangular mask of the pages).  kv_len: keys
 *           j >= kv_len[b] are masked (right padding, "Attention from Scratch"
 *           (kube-dojo), Part 3 padding mask).  A query row that sees no key
 *           outputs exact zeros (the pages raise an error for such a row; an
 *           error cannot be raised per row from a batched kernel).
 * Errors.   Every entry point returns ATTN_OK (0) or a negative code; on error
 *           attn_last_error() (per calling thread) describes it.  Nothing is
 *           printed and nothing aborts.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stdint.h>

#if defined(_WIN32)
#define ATTN_API
#else
#define ATTN_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define ATTN_F32 0
#define ATTN_BF16 1

/* Status codes. */
#define ATTN_OK 0
#define ATTN_EINVAL (-1)       /* bad argument: NULL pointer, bad size, misalignment, ... */
#define ATTN_EUNSUPPORTED (-2) /* valid request this library does not implement (never a silent fallback) */
#define ATTN_ECUDA (-3)        /* a CUDA runtime or driver call failed; see attn_last_error() */
#define ATTN_ENOMEM (-4)       /* workspace allocation failed */
#define ATTN_ETIMEOUT (-5)     /* a device-side wait hit its iteration limit (reported by attn_device_status) */
#define ATTN_ECONFLICT (-6)    /* two bf16 prefill launches shared one work counter (reported by attn_device_status) */

/*
 * attn_fwd -- prefill attention for a batch of multi-head sequences.
 *
 * Defines: "Attention from First Principles", section 5 "The full
 * multi-head computation" (scores, scale by 1/sqrt(d_head), causal mask,
 * softmax over keys, weights @ V), with the key-padding mask of "Attention
 * from Scratch" (kube-dojo), Part 3, combined by logical AND.
 *
 *   q    (B, H, Sq,  D)  query rows
 *   k    (B, H, Skv, D)  key rows
 *   v    (B, H, Skv, D)  value rows
 *   out  (B, H, Sq,  D)  written; must not overlap q, k or v
 *   scale   multiplier of Q K^T; must be finite and >= 0 (1/sqrt(D) is the
 *           pages' choice, "Why divide by the square root of the head
 *           dimension?")
 *   causal  0 or 1; causal with Sq > Skv is rejected (ATTN_EINVAL)
 *   kv_len  NULL, or device int32[B]: per-sequence valid length; keys
 *           j >= kv_len[b] are masked.  With Sq == Skv the call is
 *           self-attention over a right-padded batch and query rows
 *           i >= kv_len[b] output zeros too.  With Sq != Skv only non-causal
 *           calls take kv_len (cross-attention with a padded source,
 *           "Attention from Scratch" (kube-dojo), Part 7: the padding mask
 *           spans the source length); for a causal chunk of queries against a
 *           cache use attn_fwd_chunked.
 *   dtype   ATTN_BF16: D must be 64 or 128.  ATTN_F32: D must be 64 or 128.
 *
 * Sizes: B, H >= 1; Sq, Skv >= 0 (an empty call returns ATTN_OK and does
 * nothing); D as above; B*H*max(Sq,Skv)*D must fit in 2^31 rows of D.
 *
 * Concurrency (bf16).  The kernel hands out its work through a counter in a
 * fixed table of the library (no allocation, no clearing launch).  A direct
 * call uses the counter of its stream, so bf16 prefill calls (attn_fwd,
 * attn_fwd_gqa, attn_fwd_chunked, attn_fwd_packed, attn_fwd_host's chunks) of
 * up to 256 streams may be in flight on one device at once, any number in each;
 * a further stream takes the counter of the one that has been without a call for
 * the longest time.  A call made while its
 * stream is being captured into a CUDA graph gets a counter of its own from
 * 1024 further ones, which every replay of that graph node uses; so one
 * graph must not be replayed on two streams at the same time, nor two graphs
 * that hold captured calls 1024 apart.  A launch that finds its
 * counter in use by another launch records that in the device status word:
 * attn_device_status() then returns ATTN_ECONFLICT, and the outputs of both
 * launches are undefined.  A conflict can leave the shared counter
 * unbalanced, and so can a launch that gave up on a device-side wait
 * (ATTN_ETIMEOUT), so that later launches on it report ATTN_ECONFLICT too:
 * once no call is in flight on the device, attn_release() clears every
 * counter.
 */
ATTN_API int attn_fwd(const void *q, const void *k, const void *v, void *out, int B, int H,
                      int Sq, int Skv, int D, float scale, int causal, const int32_t *kv_len,
                      int dtype, void *stream);

/*
 * attn_fwd_gqa -- attn_fwd with grouped-query (or multi-query) attention.
 *
 * Defines: "Attention from First Principles", section 5 "The full
 * multi-head computation" and "MHA, GQA, MQA -- the KV cache lever"; "Scaled
 * dot-product attention with masking", "Grouped-query attention (GQA)": the
 * keys and values have H_kv heads, H_kv divides H, and query head h attends
 * with key/value head h / (H / H_kv) -- the head that repeating K and V
 * H / H_kv times along the head axis (repeat_interleave) puts at position h.
 * Nothing is repeated in memory.  H_kv == H is attn_fwd; H_kv == 1 is
 * multi-query attention.
 *
 *   q    (B, H,    Sq,  D)
 *   k    (B, H_kv, Skv, D)
 *   v    (B, H_kv, Skv, D)
 *   out  (B, H,    Sq,  D)  written; must not overlap q, k or v
 *
 * Every other argument, rule and error is as in attn_fwd; H_kv < 1 or H not
 * a multiple of H_kv returns ATTN_EINVAL.
 */
ATTN_API int attn_fwd_gqa(const void *q, const void *k, const void *v, void *out, int B, int H,
                          int H_kv, int Sq, int Skv, int D, float scale, int causal,
                          const int32_t *kv_len, int dtype, void *stream);

/*
 * attn_fwd_host -- attn_fwd_gqa with q, k, v, out and kv_len in HOST memory:
 * the same attention ("Attention from First Principles", section 5 "The full
 * multi-head computation"), with the copies to and from the GPU done by the
 * library and overlapped with the computation.
 *
 * The batch is cut into chunks of whole key/value-head groups (whole
 * sequences, or runs of key/value heads of one sequence), each a contiguous
 * run of (b, h) slices; chunk c is copied in while chunk c - 1 is computed
 * and chunk c - 2 is copied out, on the library's own copy streams.  Each
 * chunk is computed exactly as attn_fwd_gqa computes those slices, so the
 * result equals attn_fwd_gqa's bit for bit.
 *
 *   q, k, v, out  host pointers, layouts and sizes as in attn_fwd_gqa.  Page-
 *                 locked (pinned) memory lets the copies run asynchronously at
 *                 full speed; pageable memory works but is staged.  out must
 *                 not overlap the inputs.
 *   kv_len        NULL or HOST int32[B], meaning as in attn_fwd_gqa.
 *   stream        the work starts after work already queued on `stream`, which
 *                 resumes after the last copy out.
 *
 * Synchronous: returns when out holds the result (or on error).  D must be 64
 * or 128 (ATTN_EUNSUPPORTED otherwise).  The library keeps device copies of
 * q, k, v, out (grown on demand, freed by attn_release), so concurrent calls
 * on one device run one after the other.  Other errors as in attn_fwd_gqa;
 * ATTN_ENOMEM if the device copies cannot be allocated.
 */
ATTN_API int attn_fwd_host(const void *q, const void *k, const void *v, void *out, int B, int H,
                           int H_kv, int Sq, int Skv, int D, float scale, int causal,
                           const int32_t *kv_len, int dtype, void *stream);

/*
 * attn_fwd_chunked -- prefill of a chunk of new queries against a KV cache,
 * with the log-sum-exp of every row.
 *
 * Defines: the cache append before causal attention of "Scaled
 * dot-product attention with masking" ("The full multi-head computation":
 * past keys and values are concatenated with the new ones), with positions
 * kept absolute ("Attention from scratch" (open-llm-engineering), "KV cache
 * position drift").  Sequence b holds L_b = cache_len[b] valid cache
 * positions, the last Sq of which are the chunk's own keys and values
 * (appended by the caller); query i sits at position L_b - Sq + i and sees
 * keys j <= L_b - Sq + i.  A query whose position is negative (L_b < Sq)
 * sees no key: its row is zero.  Grouped-query heads as in attn_fwd_gqa.
 *
 *   q          (B, H,    Sq,  D)  the chunk's queries
 *   kcache     (B, H_kv, Skv, D)  cache capacity Skv >= Sq
 *   vcache     (B, H_kv, Skv, D)
 *   out        (B, H,    Sq,  D)  written; must not overlap the inputs
 *   lse        NULL, or device float (B, H, Sq), written: log(sum_j
 *              exp(scale * q_i . k_j)) over the visible keys (natural log,
 *              fp32), -inf for a row that sees none.  Not on the pages: it is
 *              what lets a caller merge attention over split key sets exactly,
 *              out = sum_c exp(lse_c - LSE) out_c with LSE = log sum_c exp(lse_c).
 *   cache_len  NULL (every L_b = Skv) or device int32[B], clamped to [0, Skv].
 *
 * dtype, D, scale, sizes and errors as in attn_fwd; Sq > Skv returns
 * ATTN_EINVAL.  With cache_len NULL and no lse this is attn_fwd_gqa with
 * causal = 1.
 */
ATTN_API int attn_fwd_chunked(const void *q, const void *kcache, const void *vcache, void *out,
                              float *lse, int B, int H, int H_kv, int Sq, int Skv, int D, float scale,
                              const int32_t *cache_len, int dtype, void *stream);

/*
 * attn_fwd_debug -- the general attention of "Attention from Scratch"
 * (kube-dojo), Part 2, for inspection: T_q != T_k, value depth d_v != d_k,
 * and the attention weights returned with the output (Part 4 "Attention
 * Maps").  One warp per query row in fp32; not a fast path.
 *
 *   q        (B, H,    Sq,  Dk)     dtype ATTN_F32 or ATTN_BF16
 *   k        (B, H_kv, Skv, Dk)
 *   v        (B, H_kv, Skv, Dv)
 *   out      (B, H,    Sq,  Dv)     written, in the input dtype
 *   weights  NULL or device float (B, H, Sq, Skv), written: the softmax
 *            weights of each row, exactly 0 for a masked key, all 0 for a
 *            row that sees no key (and for a padded query row)
 *
 * Dk, Dv in [1, 256]; Skv <= 16384 (ATTN_EUNSUPPORTED above); tensors
 * aligned to their element size.  scale, causal, kv_len, H_kv and the mask
 * rules are those of attn_fwd / attn_fwd_gqa.
 */
ATTN_API int attn_fwd_debug(const void *q, const void *k, const void *v, void *out, float *weights,
                            int B, int H, int H_kv, int Sq, int Skv, int Dk, int Dv, float scale,
                            int causal, const int32_t *kv_len, int dtype, void *stream);

/*
 * attn_decode -- one new query per (batch, head) against a KV cache.
 *
 * Defines: "Attention from First Principles", section 6 "Under the hood"
 * (decode is a matrix-vector product against the whole cache) and "Scaled
 * dot-product attention with masking", "Adding the causal mask" (with
 * seq_q = 1 the query attends to every cached position, no mask).  The
 * scale is 1/sqrt(D).
 *
 *   q       (B, H, D)        the new queries
 *   kcache  (B, H, Skv, D)   cached keys, padded to Skv
 *   vcache  (B, H, Skv, D)   cached values, padded to Skv
 *   out     (B, H, D)        written
 *   kv_len  NULL (every sequence uses all Skv positions) or device int32[B];
 *           keys j >= kv_len[b] are ignored, kv_len[b] == 0 gives zeros.
 *   dtype   ATTN_BF16 or ATTN_F32 (fp32 everywhere, on the CUDA cores); D
 *           must be 64 or 128.  All pointers 16-byte aligned.
 *
 * The kernel splits each sequence's keys into chunks processed in parallel
 * and merges the partial softmax results; the partials live in a workspace
 * the library allocates on first use (and grows when a call needs more),
 * which attn_release() frees.  The workspace is shared by all calls on a
 * device: calls that overlap in time on different streams of one device race.
 *
 * CUDA graphs: a captured call keeps the workspace's address.  Growing the
 * workspace never frees the old buffer (it is kept until attn_release), so
 * a graph captured before a larger call stays valid.  A call made during a
 * capture cannot allocate: if it needs a larger workspace than the device
 * has, it returns ATTN_EINVAL without enqueuing anything, so make one
 * ordinary call of the largest size before capturing.  Destroy every graph
 * that holds a decode call before attn_release().
 */
ATTN_API int attn_decode(const void *q, const void *kcache, const void *vcache, void *out, int B,
                         int H, int Skv, int D, const int32_t *kv_len, int dtype, void *stream);

/*
 * attn_decode_gqa -- attn_decode with grouped-query (or multi-query) attention.
 *
 * Defines: as attn_decode, with the head grouping of attn_fwd_gqa: the cache
 * has H_kv heads, H_kv divides H, and query head h attends with cached head
 * h / (H / H_kv).  One read of a cached head serves all H / H_kv query heads
 * of its group, which is why grouping raises decode's arithmetic intensity to
 * about H / H_kv flops per byte ("Attention from First Principles", section 6
 * "Under the hood").
 *
 *   q       (B, H, D)
 *   kcache  (B, H_kv, Skv, D)
 *   vcache  (B, H_kv, Skv, D)
 *   out     (B, H, D)   written
 *
 * Every other argument, rule, error and the workspace behaviour are as in
 * attn_decode; H_kv < 1 or H not a multiple of H_kv returns ATTN_EINVAL.
 * H_kv == H runs attn_decode's kernels.  In bf16, groups of G = H / H_kv >= 4
 * heads (up to 128) run on the tensor cores, the group's queries forming the
 * rows of one tile; smaller groups and fp32 run on the CUDA cores.
 */
ATTN_API int attn_decode_gqa(const void *q, const void *kcache, const void *vcache, void *out, int B,
                             int H, int H_kv, int Skv, int D, const int32_t *kv_len, int dtype,
                             void *stream);

/*
 * attn_decode_noalloc -- attn_decode that never allocates device memory.
 *
 * The pages have no counterpart: this entry point exists for callers that
 * must not allocate device memory while they run.  attn_decode allocates its
 * scratch (the per-chunk partial results) with cudaMalloc on first use and
 * whenever a call needs more; that fails or misbehaves for callers that have
 * reserved all device memory up front for their own pool (an inference server
 * sizing its KV cache to the whole GPU), and cudaMalloc / cudaFree can
 * synchronise the device, which a latency-bound decode loop cannot afford.
 * This variant runs the same kernels with the scratch in a fixed array inside
 * the library instead, so it calls no allocation routine at all.
 *
 * Arguments, layouts, dtype support and results are those of attn_decode.
 * Limit: B*H*attn_decode_splits(B,H,Skv,D)*(D + 2)*4 bytes must not exceed
 * 32 MiB (33554432); larger requests return ATTN_EINVAL with a message saying
 * how much they need (B64 H32 Skv8192 D128 needs about 17 MB).
 *
 * The array is part of the library image: every GPU that loads the library's
 * decode code holds these 32 MiB until the process exits.  The first call on
 * each device looks up the array's device address (cudaGetSymbolAddress, with
 * that device current) and caches it; make that first call before any stream
 * capture on the device.  All calls on a device share the one array and its
 * contents persist between calls (nothing in it needs to start at zero: each
 * call writes every partial it reads), so calls that overlap on the GPU (on
 * different streams, or from different threads) race and must be serialised
 * by the caller.
 */
ATTN_API int attn_decode_noalloc(const void *q, const void *kcache, const void *vcache, void *out, int B,
                                 int H, int Skv, int D, const int32_t *kv_len, int dtype, void *stream);

/*
 * attn_decode_splits -- number of KV chunks attn_decode uses per (batch,
 * head) for these sizes (for benchmarks and tests); negative on bad sizes.
 */
ATTN_API int attn_decode_splits(int B, int H, int Skv, int D);

/*
 * attn_fwd_packed -- prefill attention of sequences of different lengths packed
 * one behind the other, without padding.
 *
 * Sequence s is tokens [cu_seqlens[s], cu_seqlens[s + 1]) of token-major (T, H, D)
 * tensors, as projections write them.  Each sequence attends to itself only:
 * token i of it sees its tokens j (j <= i when causal).  Grouped heads as in
 * attn_fwd_gqa.  Rows outside every sequence (before cu_seqlens[0], from
 * cu_seqlens[n_seq] on) are left as they were in out and lse.  A key that a row
 * does not see leaves no trace in it, whatever its K and V hold: another
 * sequence's or a later token's infinities and NaNs stay theirs.  Sequences of
 * length 0 are allowed.
 *
 *   q, out    (T, H, D) rows; k, v  (T, H_kv, D) rows; out must not overlap
 *             the inputs (slices of one fused matrix do not)
 *   lse       NULL, or device float (T, H), written: the natural log-sum-exp
 *             of each row's scaled scores
 *   strides   NULL (contiguous), or HOST int64[8]: elements from token to token
 *             and from head to head of q, k, v and out, multiples of 16 bytes;
 *             pointers 16-byte aligned; rows of one tensor must not overlap
 *   cu_seqlens  device int32[n_seq + 1], nondecreasing, within [0, T].  Other
 *             contents give undefined rows of out, never an access outside
 *             the tensors.
 *   workspace   device memory of attn_fwd_packed_workspace(...) bytes, 16-byte
 *             aligned (bf16; fp32 needs none), used until the call's work on
 *             `stream` is done.  Calls that may run at the same time need one
 *             each, and a captured call keeps its address.
 *
 * Scores are held as base-2 exponents in fp32: scaled scores above 2.3e38 in
 * magnitude count as infinite.  A row whose every score is -inf is a NaN.  An
 * infinite or NaN element of V makes that element infinite or NaN in every row that
 * sees its key; where the key's weight underflows, an infinity may become a NaN.
 *
 * dtype, D, scale and errors as in attn_fwd; "Concurrency" there applies to the
 * bf16 form.  The same call gives the same bits every time.  bf16 rows do not
 * depend on what else is packed with their sequence; an fp32 row's sums are split
 * by the number of sequences and tokens, so it may differ in its last bits.
 */
ATTN_API int attn_fwd_packed(const void *q, const void *k, const void *v, void *out, float *lse, int T, int H, int H_kv,
                             int D, const long long *strides, const int32_t *cu_seqlens, int n_seq, float scale,
                             int causal, int dtype, void *workspace, long long workspace_bytes, void *stream);
/* Bytes of workspace that call needs (0 for fp32); negative on bad sizes. */
ATTN_API long long attn_fwd_packed_workspace(int T, int n_seq, int H, int H_kv, int dtype);

/*
 * attn_decode_tree -- attention of a tree of drafted tokens over a KV cache:
 * all the drafts of a speculative step in one pass over the cache.
 *
 * Sequence b has L_b = cache_len[b] valid cache rows, the last n_b =
 * draft_len[b] of them drafted tokens in tree order (attn_rope_append puts
 * them there).  Drafted token t hangs under drafted token parents[b][t] < t, or
 * under the committed cache when that is negative (or not below t).  It sees
 * the committed rows [0, L_b - n_b), its ancestors and itself.  A chain
 * (parents[t] = t - 1) is attn_fwd_chunked's causal chunk.  Rows t >= n_b, and
 * tokens whose cache row L_b - n_b + t is negative, are written as zeros.  Rows
 * that a token does not see leave no trace in it, whatever they hold.
 *
 *   q, out      (B, H, T, D) rows, T <= 128
 *   kcache, vcache  (B, H_kv, Skv, D), contiguous; H_kv divides H
 *   strides     NULL (contiguous), or HOST int64[6]: elements from sequence to
 *               sequence, head to head and token to token of q and of out,
 *               multiples of 16 bytes (a token-major (B, T, H, D) tensor is one
 *               choice)
 *   parents     device int32, T values per sequence, parents_stride apart; 0:
 *               one tree for all
 *   cache_len   device int32[B], clamped to [0, Skv], or NULL (Skv)
 *   draft_len   device int32[B], clamped to [0, T], or NULL (T)
 *   workspace   device memory of attn_decode_tree_workspace(...) bytes, 16-byte
 *               aligned (may be NULL when that is 0); rules as in attn_fwd_packed
 *
 * The splits of a sequence are merged in order: a call gives the same bits
 * every time.  bf16 cuts the work of all sequences into equal shares, so the last
 * bits of a sequence's rows may depend on the other sequences' lengths; in fp32 they
 * depend on the sizes alone.  Scores beyond fp32's range and infinite or NaN elements
 * of V as in attn_fwd_packed (which of the two a row gets where a weight underflows may
 * depend on the cuts as well).  dtype, D, scale
 * and errors as in attn_fwd; T > 128 returns ATTN_EUNSUPPORTED.
 */
ATTN_API int attn_decode_tree(const void *q, const void *kcache, const void *vcache, void *out, int B, int H, int H_kv,
                              int T, int Skv, int D, const long long *strides, const int32_t *parents,
                              int parents_stride, const int32_t *cache_len, const int32_t *draft_len, float scale,
                              int dtype, void *workspace, long long workspace_bytes, void *stream);
/* Bytes of workspace that call needs on the current device (may be 0); negative on bad sizes. */
ATTN_API long long attn_decode_tree_workspace(int B, int H, int H_kv, int T, int Skv, int D, int dtype);

/*
 * attn_fwd_paged -- attention of new tokens over a paged KV cache: chunks of prompts,
 * single tokens, and both in one call.
 *
 * The cache is a pool of pages of page_size rows; sequence s holds L_s = cache_len[s]
 * keys, key j in row j % page_size of page page_table[s][j / page_size].  Its last n_s
 * keys are those of its new tokens (attn_rope_append_paged puts them there), which are
 * tokens [cu_seqlens[s], cu_seqlens[s + 1]) of token-major (T, H, D) tensors.  Token i
 * of them sits at position L_s - n_s + i and sees keys j <= L_s - n_s + i, as in
 * attn_fwd_chunked; one whose position is negative sees none: its row is zero and its
 * lse -inf.  Grouped heads as in attn_fwd_gqa.  Rows outside every sequence (before
 * cu_seqlens[0], from cu_seqlens[n_seq] on) are left as they were in out and lse.  A key
 * that a row does not see leaves no trace in it, whatever its page holds.  Sequences may
 * share pages.
 *
 *   q, out      (T, H, D) rows; out must not overlap the inputs
 *   kpages, vpages  (n_pages, H_kv, page_size, D) pages, or any strides of them: rows of
 *               (n_pages, page_size, H_kv, D) pages, two halves of one tensor.  A
 *               contiguous (B, H_kv, Skv, D) cache is one page a sequence.
 *   page_size   a multiple of 8 (ATTN_EUNSUPPORTED otherwise); powers of two from 16 on
 *               are the fast case
 *   lse         NULL, or device float (T, H), written: the natural log-sum-exp of each
 *               row's scaled scores
 *   strides     NULL (contiguous), or HOST int64[10]: elements from token to token and
 *               from head to head of q and of out, then from page to page, head to head
 *               and row to row of kpages and of vpages; multiples of 16 bytes
 *   page_table  device int32, max_pages entries a sequence, table_stride apart.  Only
 *               entries that hold a visible key are read.  One outside [0, n_pages) counts
 *               as a page of zeros, never as an access outside the pool.
 *   cu_seqlens  device int32[n_seq + 1], nondecreasing, within [0, T], or NULL: T / n_seq
 *               tokens each (one each when T = n_seq).  Other contents give undefined
 *               rows of out and lse, never an access outside the tensors.
 *   cache_len   device int32[n_seq], each clamped to [0, max_pages * page_size], or NULL
 *               (every row of the table full)
 *   workspace   device memory of attn_fwd_paged_workspace(...) bytes, 16-byte aligned (may
 *               be NULL when that is 0); rules as in attn_fwd_packed
 *
 * The parts of a sequence are merged in order: a call gives the same bits every time.  How
 * the keys are shared out follows from the sizes of the call and, in bf16, from the lengths of
 * all sequences, so the last bits of a row may depend on those.  One of the sizes is the
 * table's width: a few short sequences in a table for many more tokens take some 5 us longer
 * than in one that fits them.  Scores beyond fp32's range and infinite or NaN elements of V as
 * in attn_decode_tree.  dtype, D, scale and errors as in attn_fwd; no work counter is used, and
 * no device memory is allocated.
 */
ATTN_API int attn_fwd_paged(const void *q, const void *kpages, const void *vpages, void *out, float *lse, int T, int H,
                            int H_kv, int D, const long long *strides, int n_pages, int page_size, const int32_t *page_table,
                            int max_pages, long long table_stride, const int32_t *cu_seqlens, const int32_t *cache_len,
                            int n_seq, float scale, int dtype, void *workspace, long long workspace_bytes, void *stream);
/* Bytes of workspace that call needs on the current device (may be 0); negative on bad
 * sizes.  ragged: cu_seqlens is given. */
ATTN_API long long attn_fwd_paged_workspace(int T, int n_seq, int H, int H_kv, int D, int max_pages, int page_size, int ragged,
                                            int dtype);

/*
 * attn_rope -- rotary positions: turns the pairs of each head row of q and k by
 * an angle proportional to the row's position, before attention or caching.
 *
 * Row element pairs are (x[p], x[p + rotary_dim/2]) (interleaved = 0) or
 * (x[2p], x[2p + 1]) (interleaved = 1), p < rotary_dim / 2; elements from
 * rotary_dim on are copied.  With n the row's position,
 *
 *     (a, b) -> mscale * (a cos(n w_p) - b sin(n w_p), b cos(n w_p) + a sin(n w_p)),
 *
 * w_p = freqs[p]; inverse = 1 turns by -n w_p, which takes a turn back and is
 * also its gradient (grad_x = mscale R(-n) grad_out).  Scaled frequencies for
 * long contexts are a matter of freqs and mscale.  Angles are formed modulo
 * one turn in 64-bit fixed point: for |w_p| < 2^40 they are off by less than 10^-9
 * radians at any position.  The fraction of a turn is then rounded to 24 bits (10^-7
 * radians); the arithmetic is fp32, rounded once to the output type.
 *
 *   q, q_out  (T, H, D) rows; k, k_out  (T, H_kv, D) rows, H_kv = 0 (and NULL)
 *             for q alone.  An output may be its own input (same pointer and
 *             strides: in place); any other overlap returns ATTN_EINVAL.
 *             Slices of one fused (T, columns) matrix do not overlap.
 *   strides   NULL (contiguous), or HOST int64[8]: elements from token to
 *             token and from head to head of q, k, q_out and k_out.  Rows of
 *             one tensor must not overlap.  (B, H, S, D) tensors are B calls, or
 *             one call when B = 1.
 *   positions device int32[T]; any value, negative ones turn backwards.
 *   freqs     HOST double[rotary_dim / 2], radians per position, finite; read
 *             during the call (a captured call keeps the values).
 *   rotary_dim  even, 0 .. D.
 *   mscale    finite multiplier of the turned elements (1 for none).
 *
 * D must be 64 or 128.  Tensors need element alignment only; 16-byte aligned
 * pointers, strides and pair offsets are the fast case.  No workspace.
 */
ATTN_API int attn_rope(const void *q, const void *k, void *q_out, void *k_out, int T, int H, int H_kv, int D,
                       const long long *strides, const int32_t *positions, const double *freqs, int rotary_dim,
                       int interleaved, int inverse, float mscale, int dtype, void *stream);

/*
 * attn_rope_append -- attn_rope of new tokens whose turned keys, and values,
 * go to their rows of a KV cache: one pass instead of a turn, two transposes
 * and two copies.  This is the append that attn_fwd_chunked, attn_decode and
 * attn_decode_tree expect of their caller, for prompts, single tokens
 * and drafts.
 *
 * Sequence b's new tokens are [cu_seqlens[b], cu_seqlens[b + 1]), n_b of them.
 * cache_len[b] = L_b counts them already (as in attn_fwd_chunked), so token i of
 * the sequence goes to cache row L_b - n_b + i, which is also its position
 * unless `positions` says otherwise (the tokens of a tree sit at their depth).
 * A token whose row is negative is turned but not cached.  Tokens outside
 * every sequence (before cu_seqlens[0], from cu_seqlens[B] on) are neither
 * read nor written anywhere.  Other cache rows stay as they were.
 *
 *   q, q_out  (T, H, D) rows; k, v  (T, H_kv, D) rows, H_kv >= 1
 *   k_out     NULL, or (T, H_kv, D) rows: the turned keys once more, token by
 *             token (attn_fwd_packed reads them); may be k itself
 *   kcache, vcache  (B, H_kv, Skv, D), contiguous, written (NULL allowed when
 *             Skv = 0: every token is turned but not cached)
 *   strides   NULL or HOST int64[10]: q, k, v, q_out, k_out, as in attn_rope
 *   cu_seqlens  device int32[B + 1], nondecreasing, or NULL: T / B tokens per
 *             sequence (T a multiple of B)
 *   cache_len device int32[B], each clamped to [0, Skv], or NULL: every L_b = Skv
 *   positions device int32[T] or NULL
 *
 * The rest as in attn_rope.
 */
ATTN_API int attn_rope_append(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *kcache,
                              void *vcache, int T, int H, int H_kv, int D, const long long *strides, int B, int Skv,
                              const int32_t *cu_seqlens, const int32_t *cache_len, const int32_t *positions,
                              const double *freqs, int rotary_dim, int interleaved, float mscale, int dtype,
                              void *stream);

/*
 * attn_norm_rope -- RMS norm of each head row of q and k, and the rotary turn of the
 * result, in one pass.
 *
 *     y = x / sqrt(mean over the row's D elements of x^2 + eps) * weight,
 *
 * then turned as attn_rope turns x.  The arithmetic is fp32 from the load to the one
 * rounding at the store (the normed row is not rounded before its turn).  The squares are
 * summed in fp32: a row of elements beyond 10^19 loses itself to their infinite sum, and
 * with eps = 0 a row of zeros is NaN.
 *
 *   q_weight, k_weight  (D,) in the call's dtype, or NULL: that tensor is turned as it is
 *   eps       finite, >= 0
 *
 * The rest as in attn_rope (outputs may be their inputs).  Fast are 16-byte aligned
 * pointers and strides with interleaved pairs or a rotary_dim / 2 of whole 16 bytes.
 */
ATTN_API int attn_norm_rope(const void *q, const void *k, void *q_out, void *k_out, int T, int H, int H_kv, int D,
                            const long long *strides, const int32_t *positions, const double *freqs, int rotary_dim,
                            int interleaved, float mscale, const void *q_weight, const void *k_weight, float eps, int dtype,
                            void *stream);

/*
 * attn_rope_append_paged -- new tokens into a paged KV cache: the norm (where weights are
 * given) and turn of attn_norm_rope, the turned keys and the values written to their pages.
 * It is the append that attn_fwd_paged expects.
 *
 * Sequence s's new tokens are [cu_seqlens[s], cu_seqlens[s + 1]), n_s of them, or T / n_seq
 * each.  cache_len[s] = L_s counts them already, so token i of the sequence is key
 * j = L_s - n_s + i, which is also its position unless `positions` says otherwise, and
 * goes to row j % page_size of page page_table[s][j / page_size].  A token whose j is
 * negative, or whose entry of the table is outside [0, n_pages), is turned but not cached.
 * Nothing is written for tokens outside every sequence; other rows of the pages stay as
 * they were.  Two tokens of a call must not have the same row of a page.
 *
 *   q, q_out  (T, H, D) rows; k, v  (T, H_kv, D) rows, H_kv >= 1
 *   k_out     NULL, or (T, H_kv, D) rows: the turned keys once more, token by token
 *   kpages, vpages  (n_pages, H_kv, page_size, D) pages, written; any page_size >= 1
 *   strides   NULL or HOST int64[16]: q, k, v, q_out, k_out as in attn_rope, then page, head
 *             and row of kpages and of vpages
 *   page_table, cu_seqlens, cache_len  as in attn_fwd_paged
 *   positions device int32[T] or NULL
 *
 * The rest as in attn_norm_rope.
 */
ATTN_API int attn_rope_append_paged(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *kpages,
                                    void *vpages, int T, int H, int H_kv, int D, const long long *strides, int n_pages,
                                    int page_size, const int32_t *page_table, int max_pages, long long table_stride,
                                    const int32_t *cu_seqlens, const int32_t *cache_len, int n_seq, const int32_t *positions,
                                    const double *freqs, int rotary_dim, int interleaved, float mscale, const void *q_weight,
                                    const void *k_weight, float eps, int dtype, void *stream);

/*
 * attn_pages_step -- the next table of pages: sequences grow, are cut back, fork, end and
 * begin, without the host.
 *
 * Row b of the new table goes on from row parents[b] of the old one (several rows may have
 * one parent: they fork; a parent outside [0, n_seq) starts an empty sequence; a row that
 * nobody goes on from has ended).  It is to hold new_len[b] tokens, of which it keeps the
 * first keep = min(cache_len[parents[b]], new_len[b]) of its parent's:
 *   - The keep / page_size full pages are shared with whoever else holds them.
 *   - A partly filled page, to whose rows behind `keep` the sequence will append, has one
 *     holder: the lowest row that keeps it so, unless some row keeps it full or it is
 *     pinned.  Every other row gets a new page and asks for a copy of its rows.
 *   - Entries up to ceil(new_len[b] / page_size) that are missing, or are no pages, become
 *     new pages; entries from there on are -1.
 * New pages are those that no row of the new table keeps and that are not pinned, the
 * lowest first, given out in the order of rows and of entries.  A page that ends with its
 * sequence can be given out in the same call.  Where they run out, entries are -1 (tokens
 * there are not cached, their keys read as zeros; a fork's copy is not asked for) and
 * free_pages is negative.  A later call gives such an entry a page, but not the tokens that
 * were to be in it: its rows are whatever they were.  So a negative free_pages is an answer
 * to act on before anything is appended.  Until the copies are made nothing has moved, and
 * a call from the old table with fewer or shorter rows has all their tokens.  Or the copies
 * are made, and a call from the new table cuts each row back to its entries in front of
 * the first -1.
 *
 *   page_table  device int32 (n_seq, max_pages), rows table_stride apart
 *   cache_len   device int32[n_seq], each clamped to [0, max_pages * page_size], or NULL
 *               (every row full)
 *   parents     device int32[n_out], or NULL: row b goes on from row b (n_out = n_seq)
 *   new_len     device int32[n_out], clamped like cache_len, or NULL: the parent's length
 *   pinned      device int32[n_pages] or NULL: pages with a value other than 0 are held
 *               outside the table too (a cache of prefixes): never given out, never written
 *   table_out   (n_out, max_pages), rows out_stride apart, written; len_out (n_out): the
 *               clamped new_len; copies (n_out, 3): page copied from, page copied to and
 *               rows, or -1, -1, 0 where the row needs none (for attn_pages_copy, before
 *               anything is appended); free_pages (1): free pages left, or minus those
 *               missing.  Outputs must not overlap inputs.
 *   workspace   device memory of attn_pages_workspace(n_out, n_pages) bytes, 16-byte
 *               aligned; rules as in attn_fwd_packed
 *
 * n_out is at most 2^29, n_out max_pages and n_pages are below 2^30.  The same call gives the
 * same table every time.
 */
ATTN_API int attn_pages_step(const int32_t *page_table, const int32_t *cache_len, int n_seq, int max_pages, long long table_stride,
                             int n_pages, int page_size, const int32_t *parents, const int32_t *new_len,
                             const int32_t *pinned, int n_out, int32_t *table_out, long long out_stride, int32_t *len_out,
                             int32_t *copies, int32_t *free_pages, void *workspace, long long workspace_bytes,
                             void *stream);
/* Bytes of workspace of attn_pages_step and attn_pages_compact (n_out = n_seq there). */
ATTN_API long long attn_pages_workspace(int n_out, int n_pages);

/*
 * attn_pages_compact -- moves the pages held together at the front of the pool.
 *
 * With n pages held (by the rows up to cache_len, or pinned), the k-th lowest page from n
 * on that a row holds and that is not pinned becomes the k-th lowest free page below n, in
 * every row that holds it.  table_out names the new places (-1 behind a row's pages and for
 * entries that are no pages); copies ((n_pages + 1) / 2, 3) lists page copied from, page
 * copied to and page_size, then -1, -1, 0; free_pages (1) is n_pages - n.  Arguments
 * as in attn_pages_step.
 */
ATTN_API int attn_pages_compact(const int32_t *page_table, const int32_t *cache_len, int n_seq, int max_pages,
                                long long table_stride, int n_pages, int page_size, const int32_t *pinned, int32_t *table_out,
                                long long out_stride, int32_t *copies, int32_t *free_pages, void *workspace,
                                long long workspace_bytes, void *stream);

/*
 * attn_pages_copy -- copies of pages, keys and values of all layers: for each (from, to,
 * rows) of `copies` the first `rows` rows of page `to` become those of page `from`.
 *
 *   kpages, vpages  (layers, n_pages, H_kv, page_size, D) pages, any strides; not
 *             overlapping each other
 *   strides   NULL (contiguous), or HOST int64[8]: layer, page, head and row of kpages and
 *             of vpages in elements.  16-byte aligned pointers and strides are the fast case.
 *   copies    device int32 (n_copies, 3), at most 2^29.  Pairs with a page outside [0, n_pages) are
 *             passed over, rows are clamped to [0, page_size].  A page that one pair writes
 *             must not be read or written by another (the lists of attn_pages_step and
 *             attn_pages_compact are such).  A pair passed over costs some 2 ns a layer: of a
 *             compaction's list, whose pairs come first, the first so many may be given.
 */
ATTN_API int attn_pages_copy(void *kpages, void *vpages, int layers, int n_pages, int H_kv, int page_size, int D,
                             const long long *strides, const int32_t *copies, int n_copies, int dtype, void *stream);

/*
 * attn_device_status -- synchronise `stream`, then report and clear the
 * device-side status word.  Returns ATTN_OK, ATTN_ETIMEOUT when a kernel gave
 * up on a device-side wait (its output is then undefined), ATTN_ECONFLICT
 * when two bf16 prefill launches in flight shared one work counter (see
 * attn_fwd, "Concurrency"; both outputs are undefined), or ATTN_ECUDA when
 * the synchronisation itself failed.
 */
ATTN_API int attn_device_status(void *stream);

/*
 * attn_selftest_wait_timeout -- diagnostic: enqueue a one-warp kernel whose
 * only device-side wait can never complete, with a limit of `limit_cycles` SM
 * clock cycles (0 .. 2e9).  The wait gives up, the kernel records the timeout
 * in the device status word and exits, so the next attn_device_status(stream)
 * returns ATTN_ETIMEOUT (and clears the word).  Used to check, on a real
 * device and without any fault or hang, the path every kernel's bounded waits
 * take when a logic error would otherwise deadlock.  There is no counterpart
 * on the pages.
 */
ATTN_API int attn_selftest_wait_timeout(long long limit_cycles, void *stream);

/* Description of the last error on the calling thread ("" if none). */
ATTN_API const char *attn_last_error(void);

/* Free library-owned device memory on the current device: the decode
 * workspace (with every smaller buffer it replaced) and attn_fwd_host's
 * device copies; and clear the bf16 prefill work counters (the recovery after
 * ATTN_ECONFLICT).  Not while any call of the library is running on the
 * device, and not while a CUDA graph that holds a library call may still be
 * replayed. */
ATTN_API void attn_release(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
