// fp32 attention over tiles on the CUDA cores (FFMA only, no TF32): packed
// sequences (attn_fwd_packed), trees of drafted tokens (attn_decode_tree) and new
// tokens over a paged cache (attn_fwd_paged).
//
// 32 query rows against tiles of 32 keys, online softmax in log2 units.  A warp
// holds 16 rows x 32 keys of scores as 4 x 4 a thread (rows ty + 4 i, keys tx + 8 j)
// and 16 x D of output as 4 rows x D / 8 columns a thread.  FMAs go in pairs (two
// depths of a score, two columns of the output).  The eight lanes that share rows
// differ in bits 1-3 of their number: then lanes 2 l and 2 l + 1 read the same K and V
// elements, lanes l and l ^ 2 the same Q and P elements, and a 16-byte shared-memory
// load takes two passes instead of four (passes of the whole kernel 5.6 to 3.4 million).
// K rows are padded by 16 bytes so that eight lanes read
// eight rows without conflicts.  The next tile's K is copied in (cp.async) while P V
// runs, its V while the scores are computed.
//
// Few rows and long keys leave one warp per scheduler waiting on shared memory
// and shuffles, so a block has several workers, pairs of warps, that share the keys of
// the same rows equally (in units of 8) and join their output, max and sum at the end:
// as many as shared memory holds, which also means one block an SM, so that a block
// left over goes to the SM that is done first and not beside a long one; or half as
// many and two blocks an SM, where there are many blocks (the launches say when).
//
// Measured: six sequences of 700 to 1 tokens, 4 heads of depth 64, not causal (0.86
// GFLOP, 11.6 us of FMAs): 39.5 us.  No pipe bounds it: 232 blocks on 152 SMs leave a
// second round to some of the long ones (a third of the SMs' time idle), and while an SM
// has work the FMA pipe (51 %), the issue slots (50 %) and shared memory (48 %) are each
// half busy, 16 warps that wait on the FMA pipe in turn, on results and on the three
// barriers of a tile.
// Earlier forms, 128 threads a tile of 64 keys: one a block 90 us, two 47 us, four 43
// us, with equal shares 40 us; 8 rows a thread 45 us.
//
// Single tokens over pages leave most of the 32 rows empty: with up to four, only the
// first row of a thread is computed (64 tokens over 2000 keys, H 8 / 2, D 64: 39 against
// 76 us), a split of the keys may be as short as a unit for each worker (six
// sequences of up to 1024 keys and two chunks: 11.0 us, with 64 keys at least and all rows
// 14.7), and the entries of the table are looked up once a unit, not once a copy (34 and 10.7
// us; 64 tokens over 2000 keys, H 8 / 8, D 128, 1.05 GB: 220 us, 4.8 TB/s, against 310).
//
// Packed rows: a block's 32 rows lie in one sequence (a block that straddled two
// would walk the keys of both), found by a search, not a table: sequence s
// owns the blocks from cu[s] / 32 + s on, a few of which stay empty.  Tree rows
// see [0, hi) and the draft keys in their ancestor set.  A key that a row does
// not see contributes nothing whatever its row of V holds.
#include "clusters.cuh"
#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"
#include "serving.cuh"

#include <math.h>
#include <type_traits>

namespace attn {
namespace {

constexpr int kRows = 32;        // of a block
constexpr int kKeys = 32;        // of a tile
// W workers (pairs of warps) a block: kMany<D> fill an SM's shared memory, half of them
// leave room for a second block.
template <int D>
constexpr int kMany = D == 64 ? 8 : 4;
template <int W>
constexpr int kThreads = W * 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int W>
struct F32Smem {
    float q[kRows][D + 4];
    struct {
        float k[kKeys][D + 4];
        float v[kKeys][D];       // after the walk: the worker's output, [kRows][D]
        float p[2][kRows / 2][kKeys + 8];
    } w[W];
    float2 ml[W][kRows];  // each worker's max and sum
    float4 joined[kRows * D / 4];   // this CTA's part, read by the first CTA of its cluster
    float2 joined_ml[kRows];
    Ancestors anc;
};
static_assert(kRows == kKeys, "a worker's output takes its V tile's place");

// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Running state of a thread's four rows, row(i): columns 32 c + 4 tx + e, in pairs.
template <int D>
struct Rows4 {
    float m[4], l[4];
    uint64_t o[4][D / 16];
};
// Lane l is thread (tx, ty): bits 0 and 4 of l are ty, the others tx.
__device__ __forceinline__ int tx_of() { return static_cast<int>(threadIdx.x / 2 % 8); }
__device__ __forceinline__ int ty_of() { return static_cast<int>(threadIdx.x % 2 + threadIdx.x / 16 % 2 * 2); }
__device__ __forceinline__ int row_of(int i) { return static_cast<int>(threadIdx.x / 32 % 2) * (kRows / 2) + ty_of() + 4 * i; }

// This worker's part of keys [k0, k1), an equal share in units of 8 keys (the whole
// block calls it, with the copies of Q committed as one group): K row j at kat(j, in),
// V row j at vat(j, in), an address to be read where `in` is true.  visible(i, key0)
// gives the bits of keys key0 + tx + 8 j, j < 4, of row_of(i).  A warp none of whose rows is used
// (`active` is false) only copies and keeps step.
// Paged: k0 is a multiple of 8, kat and vat give a unit's first row, its stride and whether it may
// be read; where `few` is set only the first of a thread's rows is used (a block of up to four).
template <int D, int W, bool Paged = false, typename KAt, typename VAt, typename Visible>
__device__ __forceinline__ void walk(F32Smem<D, W> &smem, KAt kat, VAt vat, int k0, int k1, float sl2, bool active,
                                     Rows4<D> &st, Visible visible, bool few = false) {
    const int worker = threadIdx.x / 64, tid = threadIdx.x % 64, half = tid / 32, tx = tx_of(), ty = ty_of();
    auto &sm = smem.w[worker];
    auto &sp = sm.p[half];
    const auto sync = [&] { named_bar_sync(1 + worker, 64); };
    constexpr int C = D / 32;
    const int per = (max(k1 - k0, 0) + 8 * W - 1) / (8 * W) * 8;
    const int first = k0 + worker * per, last = min(first + per, k1);  // no keys if last <= first
    // the key units of 8 in the tile at key0; rows past the last key are zeros
    auto units = [&](int key0) { return min((last - key0 + 7) / 8, kKeys / 8); };
    auto load = [&](float *dst, int stride, auto at, int key0) {
        const uint32_t to = smem_u32(dst);
        if constexpr (Paged) {  // a unit lies in one page: looked up once
            const int n = units(key0);
#pragma unroll
            for (int u = 0; u < kKeys / 8; ++u) {
                if (u >= n) break;
                const auto page = at(key0 + 8 * u);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int row = i * (256 / D) + tid / (D / 4), c = tid % (D / 4);
                    const bool in = page.in && key0 + 8 * u + row < last;
                    cp_async16(to + ((8 * u + row) * stride + 4 * c) * 4, page.row + (in ? row * page.stride : 0) + 4 * c, in ? 16u : 0u);
                }
            }
        } else {
            const int n = units(key0) * (8 * D / 4);
#pragma unroll 8
            for (int i = tid; i < n; i += 64) {
                const int row = i / (D / 4), c = i % (D / 4);
                const bool in = key0 + row < last;
                cp_async16(to + (row * stride + 4 * c) * 4, at(key0 + row, in) + 4 * c, in ? 16u : 0u);
            }
        }
        cp_async_commit();
    };
    if (first < last) {
        load(&sm.k[0][0], D + 4, kat, first);
        load(&sm.v[0][0], D, vat, first);
        cp_async_wait<2>();  // Q, copied in before by the whole block
    } else {
        cp_async_wait<0>();
    }
    __syncthreads();
    for (int key0 = first; key0 < last; key0 += kKeys) {
        const bool more = key0 + kKeys < last;
        const int n_units = units(key0);
        cp_async_wait<1>();  // K of this tile (V may still be on its way)
        sync();
        bool hidden = false;  // a row of the thread misses a key of the tile (those past k1 are zeros)
        auto score = [&](auto n, auto rows) {
            constexpr int N = decltype(n)::value, R = decltype(rows)::value;
            uint64_t s2[R][N] = {};  // sums over even and over odd depths
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                ulonglong2 qa[R], kb[N];
#pragma unroll
                for (int i = 0; i < R; ++i) qa[i] = *reinterpret_cast<const ulonglong2 *>(&smem.q[row_of(i)][d]);
#pragma unroll
                for (int j = 0; j < N; ++j) kb[j] = *reinterpret_cast<const ulonglong2 *>(&sm.k[tx + 8 * j][d]);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        s2[i][j] = ffma2(qa[i].x, kb[j].x, s2[i][j]);
                        s2[i][j] = ffma2(qa[i].y, kb[j].y, s2[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const uint32_t see = visible(i, key0);
                float s[N], mt = -INFINITY;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    // rounded before the difference below: huge scores
                    s[j] = __fmul_rn(f2_lo(s2[i][j]) + f2_hi(s2[i][j]), sl2);
                    hidden = hidden || (!(see >> j & 1u) && key0 + tx + 8 * j < k1);
                    if (see >> j & 1u) mt = fmaxf(mt, s[j]);
                }
#pragma unroll
                for (int x = 2; x < 16; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
                const float mn = fmaxf(st.m[i], mt);
                const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet (or nothing but -inf)
                const float corr = ex2_approx(st.m[i] - ref);
                st.m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    // A seen key's weight is never 0, however far it lies below the others: an
                    // infinite or NaN value of it stays in the row (2^-149 of a finite one is
                    // less than the 2^-126 that ex2 flushes).  Marking unseen keys instead, by
                    // -0 or a mask in the product below, cost 1-5 %.
                    const float p = see >> j & 1u ? max_nan(ex2_approx(s[j] - ref), 0x1p-149f) : 0.f;
                    sum += p;
                    sp[ty + 4 * i][tx + 8 * j] = p;
                }
                st.l[i] = st.l[i] * corr + sum;  // this thread's keys; summed over the eight lanes at the end
                const uint64_t corr2 = f2_pack(corr, corr);
#pragma unroll
                for (int e = 0; e < 2 * C; ++e) st.o[i][e] = fmul2(st.o[i][e], corr2);
            }
        };
        auto score_units = [&](auto rows) {
            if (n_units == 4)
                score(std::integral_constant<int, 4>{}, rows);
            else if (n_units == 3)
                score(std::integral_constant<int, 3>{}, rows);
            else if (n_units == 2)
                score(std::integral_constant<int, 2>{}, rows);
            else
                score(std::integral_constant<int, 1>{}, rows);
        };
        if (!active) {
        } else if (Paged && few)
            score_units(std::integral_constant<int, 1>{});
        else
            score_units(std::integral_constant<int, 4>{});
        // every row of the warp sees every key: plain FMAs; otherwise a weight of zero, that
        // of a key the row does not see, must not meet an infinite or NaN value
        const bool edge = __any_sync(0xffffffffu, hidden);
        cp_async_wait<0>();  // V of this tile
        sync();              // both warps are done with K; V and P are visible
        if (more) load(&sm.k[0][0], D + 4, kat, key0 + kKeys);
        auto mix = [&](auto guarded, auto rows) {
            constexpr int R = decltype(rows)::value;
#pragma unroll 1
            for (int j = 0; j < 8 * n_units; j += 4) {
                float4 p4[R];
#pragma unroll
                for (int i = 0; i < R; ++i) p4[i] = *reinterpret_cast<const float4 *>(&sp[ty + 4 * i][j]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    uint64_t p2[R];
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float p = jj == 0 ? p4[i].x : jj == 1 ? p4[i].y : jj == 2 ? p4[i].z : p4[i].w;
                        p2[i] = f2_pack(p, p);
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&sm.v[j + jj][32 * c + 4 * tx]);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const uint64_t a = ffma2(p2[i], x.x, st.o[i][2 * c]), b = ffma2(p2[i], x.y, st.o[i][2 * c + 1]);
                            if (!decltype(guarded)::value || f2_lo(p2[i]) != 0.f) {
                                st.o[i][2 * c] = a;
                                st.o[i][2 * c + 1] = b;
                            }
                        }
                    }
                }
            }
        };
        if (!active) {
        } else if (Paged && few)
            mix(std::true_type{}, std::integral_constant<int, 1>{});
        else if (edge)
            mix(std::true_type{}, std::integral_constant<int, 4>{});
        else
            mix(std::false_type{}, std::integral_constant<int, 4>{});
        sync();  // V and P are free
        if (more) load(&sm.v[0][0], D, vat, key0 + kKeys);
    }
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 2; x < 16; x <<= 1) st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], x);
}

// Rows gs elements apart; k0 is one that may be read.
__device__ __forceinline__ auto rows_at(const float *base, long long gs, int k0) {
    return [=](int key, bool in) { return base + (in ? key : k0) * gs; };
}

template <int D>
__device__ __forceinline__ void reset(Rows4<D> &st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        st.m[i] = -INFINITY;
        st.l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st.o[i][e] = 0;
    }
}

// The workers' parts of one row, joined in order: thread t holds C float4 of row
// t / kLanes, columns 4 (t % kLanes + kLanes c).
template <int D, int W>
struct Joined {
    static constexpr int kLanes = kThreads<W> / kRows, C = D / 4 / kLanes;
    float m, l;
    float4 o[C];
    static __device__ __forceinline__ int row() { return static_cast<int>(threadIdx.x) / kLanes; }
    static __device__ __forceinline__ int column(int c) { return 4 * (static_cast<int>(threadIdx.x) % kLanes + kLanes * c); }
    __device__ __forceinline__ float4 times(int c, float f) const {
        return make_float4(o[c].x * f, o[c].y * f, o[c].z * f, o[c].w * f);
    }
};

// The whole block calls it.
template <int D, int W>
__device__ __forceinline__ Joined<D, W> join_workers(F32Smem<D, W> &sm, const Rows4<D> &st) {
    using J = Joined<D, W>;
    const int worker = threadIdx.x / 64, tx = tx_of();
    float *po = &sm.w[worker].v[0][0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (tx == 0) sm.ml[worker][row_of(i)] = make_float2(st.m[i], st.l[i]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            *reinterpret_cast<ulonglong2 *>(po + row_of(i) * D + 32 * c + 4 * tx) =
                make_ulonglong2(st.o[i][2 * c], st.o[i][2 * c + 1]);
    }
    __syncthreads();
    J r;
    r.m = -INFINITY;
    r.l = 0.f;
    float2 ml[W];
#pragma unroll
    for (int y = 0; y < W; ++y) {
        ml[y] = sm.ml[y][J::row()];
        r.m = fmaxf(r.m, ml[y].x);
    }
    const float ref = r.m == -INFINITY ? 0.f : r.m;
#pragma unroll
    for (int c = 0; c < J::C; ++c) r.o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < W; ++y) {
        const float w = ex2_approx(ml[y].x - ref);
        r.l = fmaf(w, ml[y].y, r.l);
#pragma unroll
        for (int c = 0; c < J::C; ++c) {
            const float4 x = *reinterpret_cast<const float4 *>(&sm.w[y].v[J::row()][J::column(c)]);
            r.o[c] = make_float4(fmaf(w, x.x, r.o[c].x), fmaf(w, x.y, r.o[c].y), fmaf(w, x.z, r.o[c].z), fmaf(w, x.w, r.o[c].w));
        }
    }
    return r;
}

// The cluster's parts into those of its first CTA, in order of the keys; returns
// whether this CTA is the one that holds the result.  Every thread calls it.
template <int D, int W>
__device__ __forceinline__ bool join_cluster(F32Smem<D, W> &sm, Joined<D, W> &x) {
    using J = Joined<D, W>;
    const unsigned n = cluster_size(), rank = cluster_rank();
    if (n == 1) return true;
    const int tid = threadIdx.x;
    if (rank > 0) {
#pragma unroll
        for (int c = 0; c < J::C; ++c) sm.joined[c * kThreads<W> + tid] = x.o[c];
        if (tid % J::kLanes == 0) sm.joined_ml[J::row()] = make_float2(x.m, x.l);
    }
    cluster_sync();
    if (rank == 0) {
#pragma unroll 1
        for (unsigned y = 1; y < n; ++y) {
            float m, l;
            float4 o[J::C];
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(m), "=f"(l)
                         : "r"(map_rank(&sm.joined_ml[J::row()], y)));
#pragma unroll
            for (int c = 0; c < J::C; ++c)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(o[c].x), "=f"(o[c].y), "=f"(o[c].z), "=f"(o[c].w)
                             : "r"(map_rank(&sm.joined[c * kThreads<W> + tid], y)));
            const float mn = fmaxf(x.m, m), ref = mn == -INFINITY ? 0.f : mn;
            const float w0 = ex2_approx(x.m - ref), w1 = ex2_approx(m - ref);
            x.m = mn;
            x.l = fmaf(w1, l, x.l * w0);
#pragma unroll
            for (int c = 0; c < J::C; ++c)
                x.o[c] = make_float4(fmaf(w1, o[c].x, x.o[c].x * w0), fmaf(w1, o[c].y, x.o[c].y * w0),
                                     fmaf(w1, o[c].z, x.o[c].z * w0), fmaf(w1, o[c].w, x.o[c].w * w0));
        }
    }
    cluster_sync();  // the parts have been read
    return rank == 0;
}

// ------------------------------------------------------------ packed sequences

// Number of sequences whose first block, cu[s] / kRows + s, is <= w (32 probes a step).
__device__ __forceinline__ int blocks_le(const int32_t *cu, int n, int w, int T, int lane) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, at < hi && min(max(cu[at], 0), T) / kRows + at <= w);
        const int c = le == 0xffffffffu ? 32 : __ffs(~le) - 1;
        if (c == 0) break;
        hi = min(hi, lo + c * step);
        lo = lo + (c - 1) * step + 1;
    }
    return lo;
}

// Cluster (h, w): head h, 32 rows of the sequence that owns w.
template <int D, int W>
__global__ void __launch_bounds__(kThreads<W>, W == kMany<D> ? 1 : 2) packed_f32_kernel(const PackedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t f32_smem[];
    F32Smem<D, W> &sm = *reinterpret_cast<F32Smem<D, W> *>(f32_smem);
    const int tid = threadIdx.x, tx = tx_of();
    const unsigned n_cta = cluster_size(), x = blockIdx.x / n_cta;
    const int h = x % a.H, w = x / a.H, g = h / (a.H / a.H_kv);
    const int s = blocks_le(a.cu_seqlens, a.B, w, a.Sq, tid % 32) - 1;
    if (s < 0) return;  // as every CTA of the cluster
    const int c0 = min(max(a.cu_seqlens[s], 0), a.Sq), c1 = min(max(a.cu_seqlens[s + 1], c0), a.Sq);
    const int t0 = c0 + (w - c0 / kRows - s) * kRows;  // first row
    if (t0 >= c1) return;                              // one of the empty blocks
    const int end = min(t0 + kRows, c1);
    const float *Q = static_cast<const float *>(a.q) + h * a.q_hs;
    for (int i = tid; i < kRows * D / 4; i += kThreads<W>) {
        const int r = i / (D / 4), c = i % (D / 4);
        const bool in = t0 + r < end;
        cp_async16(smem_u32(&sm.q[r][4 * c]), Q + (in ? t0 + r : t0) * a.q_ts + 4 * c, in ? 16u : 0u);
    }
    cp_async_commit();
    const int limit = a.causal ? end : c1;
    int hi[4];  // rows see keys [c0, hi)
#pragma unroll
    for (int i = 0; i < 4; ++i) hi[i] = a.causal ? min(t0 + row_of(i) + 1, limit) : limit;
    // this CTA's share of the keys, in units of 8
    const int share = (limit - c0 + 8 * static_cast<int>(n_cta) - 1) / (8 * static_cast<int>(n_cta)) * 8;
    const int k0 = min(c0 + static_cast<int>(cluster_rank()) * share, limit), k1 = min(k0 + share, limit);
    Rows4<D> st;
    reset(st);
    walk<D, W>(sm, rows_at(static_cast<const float *>(a.k) + g * a.k_hs, a.k_ts, k0),
            rows_at(static_cast<const float *>(a.v) + g * a.v_hs, a.v_ts, k0), k0, k1, a.scale * kLog2e, t0 + tid / 32 % 2 * (kRows / 2) < end, st, [&](int i, int key0) {
                uint32_t see = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) see |= (key0 + tx + 8 * j < hi[i] ? 1u : 0u) << j;
                return see;
            });
    Joined<D, W> y = join_workers(sm, st);
    if (!join_cluster(sm, y)) return;
    const long long t = t0 + y.row();
    if (t >= end) return;
    const float inv = 1.f / y.l;
    float *O = static_cast<float *>(a.out) + t * a.o_ts + h * a.o_hs;
#pragma unroll
    for (int c = 0; c < y.C; ++c) *reinterpret_cast<float4 *>(O + y.column(c)) = y.times(c, inv);
    if (a.lse && y.column(0) == 0) a.lse[t * a.H + h] = (y.m + log2f(y.l)) * kLn2;
}

template <int D, int W>
cudaError_t launch_packed_f32_w(const PackedArgs &a) {
    const size_t smem = sizeof(F32Smem<D, W>);
    cudaError_t e = cudaFuncSetAttribute(packed_f32_kernel<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const long long blocks = packed_f32_blocks(a.Sq, a.B) * a.H, sms = a.n_sm > 0 ? a.n_sm : 1;
    // Fewer blocks than SMs: clusters of CTAs share the keys, 64 and more each at the mean
    // length (300 and 200 tokens, 4 heads: 14.6 us without, 10.5 with).  More blocks than
    // that lose by it: 232 blocks as 464 CTAs 41.3 against 39.8 us, 260 as 520 134 against
    // 123 us.
    unsigned cluster = 1;
    while (cluster < 8 && blocks * cluster <= sms && a.Sq / a.B >= 128 * static_cast<int>(cluster)) cluster *= 2;
    return launch_clusters(packed_f32_kernel<D, W>, cluster, static_cast<unsigned>(blocks * cluster), kThreads<W>, smem, a.stream, a);
}

template <int D>
cudaError_t launch_packed_f32_t(const PackedArgs &a) {
    // Many short blocks: two of half the workers an SM hide each other's start and end (40
    // sequences of 128 tokens, 4 heads 28 against 37 us; 20 of 400 97 against 111); few
    // or long ones are spread more evenly by one (700 to 1 tokens 39 against 47 us, one
    // of 2048 123 against 128).  Between them: as many blocks an SM as 128-key
    // stretches in the mean sequence.
    const long long blocks = packed_f32_blocks(a.Sq, a.B) * a.H, mean = a.Sq / a.B;
    const bool small = blocks > a.n_sm && blocks * 128 >= mean * a.n_sm;
    return small ? launch_packed_f32_w<D, kMany<D> / 2>(a) : launch_packed_f32_w<D, kMany<D>>(a);
}

// ------------------------------------------------------------ trees of drafted tokens

// Block x: (sequence and key/value head, 32 rows, split of the cache).  Up to eight
// splits are a cluster, whose first CTA writes the result; more leave their parts in
// the workspace.
template <int D, int W>
__global__ void __launch_bounds__(kThreads<W>, W == kMany<D> ? 1 : 2) tree_f32_kernel(const TreeArgs a, const int row_tiles) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t f32_smem[];
    F32Smem<D, W> &sm = *reinterpret_cast<F32Smem<D, W> *>(f32_smem);
    const int tid = threadIdx.x, tx = tx_of();
    const bool cluster = a.n_split <= kTreeClusterF32;  // of a.n_split CTAs
    const int c = blockIdx.x % a.n_split, m = blockIdx.x / a.n_split % row_tiles;
    const int bk = blockIdx.x / a.n_split / row_tiles, b = bk / a.H_kv, g = bk % a.H_kv;
    const int G = a.H / a.H_kv, rows = G * a.T, r0 = m * kRows;
    const Draft d = draft_of(a, b);
    const int k0 = c * a.chunk, k1 = min(k0 + a.chunk, d.L);
    if (k0 >= k1 && !cluster) return;  // the merge never reads this split
    for (int i = tid; i < kRows * D / 4; i += kThreads<W>) {
        const int r = r0 + i / (D / 4), col = 4 * (i % (D / 4));
        const bool in = r < rows && r % a.T < d.n;
        const float *q = static_cast<const float *>(a.q);
        if (in) q += b * a.q_bs + (g * G + r / a.T) * a.q_hs + (r % a.T) * a.q_ts + col;
        cp_async16(smem_u32(&sm.q[i / (D / 4)][col]), q, in ? 16u : 0u);
    }
    cp_async_commit();
    if (tid < 128) build_ancestors<128>(a, b, d, sm.anc, tid, [] { named_bar_sync(1, 128); });
    bool live[4];
    const uint32_t *w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + row_of(i), t = r % a.T;
        live[i] = r < rows && t < d.n && d.past + t >= 0;
        w[i] = sm.anc.bits[t];
    }
    Rows4<D> st;
    reset(st);
    const size_t head = static_cast<size_t>(bk) * a.Skv * D;
    if (k0 < k1) {
        walk<D, W>(sm, rows_at(static_cast<const float *>(a.k) + head, D, k0),
                rows_at(static_cast<const float *>(a.v) + head, D, k0), k0, k1, a.scale * kLog2e, __any_sync(0xffffffffu, live[0] || live[1] || live[2] || live[3]), st, [&](int i, int key0) {
                    uint32_t see = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        see |= (visible32(w[i], key0 + 8 * j + tx - d.past) & 1u) << j;
                    return live[i] ? see : 0u;
                });
    } else {
        cp_async_wait<0>();
    }
    Joined<D, W> x = join_workers(sm, st);
    if (cluster && !join_cluster(sm, x)) return;
    const int r = r0 + x.row(), t = r % a.T;
    if (r >= rows) return;
    float *O;
    float f = 1.f;
    if (cluster) {
        O = static_cast<float *>(a.out) + b * a.o_bs + (g * G + r / a.T) * a.o_hs + t * a.o_ts;
        f = t < d.n && d.past + t >= 0 ? 1.f / x.l : 0.f;
    } else {
        const size_t part = (static_cast<size_t>(bk) * rows + r) * a.n_split + c;
        O = a.part_o + part * D;
        if (x.column(0) == 0) *reinterpret_cast<float2 *>(a.part_ml + part * 2) = make_float2(x.m, x.l);
    }
#pragma unroll
    for (int cc = 0; cc < x.C; ++cc) *reinterpret_cast<float4 *>(O + x.column(cc)) = x.times(cc, f);
}

template <int D, int W>
cudaError_t launch_tree_f32_w(const TreeArgs &a) {
    const size_t smem = sizeof(F32Smem<D, W>);
    cudaError_t e = cudaFuncSetAttribute(tree_f32_kernel<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int row_tiles = ((a.H / a.H_kv) * a.T + kRows - 1) / kRows;
    const unsigned grid = static_cast<unsigned>(a.B * a.H_kv) * a.n_split * row_tiles;
    const bool cluster = a.n_split <= kTreeClusterF32;
    e = launch_clusters(tree_f32_kernel<D, W>, cluster ? static_cast<unsigned>(a.n_split) : 1u, grid, kThreads<W>, smem,
                        a.stream, a, row_tiles);
    if (e != cudaSuccess || cluster) return e;
    return launch_tree_merge_f32(a);
}

template <int D>
cudaError_t launch_tree_f32_t(const TreeArgs &a) {
    const long long blocks = static_cast<long long>(a.B) * a.H_kv * a.n_split * (((a.H / a.H_kv) * a.T + kRows - 1) / kRows);
    // more blocks than SMs: two an SM (8 sequences of 1024 rows, 32 drafts, H 8, H_kv 2: 32
    // against 54 us; 64 of 500 rows, 4 drafts, H 8, H_kv 8: 67 against 105)
    return blocks > a.n_sm ? launch_tree_f32_w<D, kMany<D> / 2>(a) : launch_tree_f32_w<D, kMany<D>>(a);
}

// ------------------------------------------------------------ new tokens over a paged cache

// The 32 rows of a block: rows [r0, r0 + 32) of a sequence's n G (token by token, row r is
// token r / G, head r % G), and the keys [0, keys) that the last of them sees.
struct PagedBlock {
    int s, c0, n, past, r0, keys;
};
// Block w of any cached head; n = 0: an empty one.  The whole warp calls it.
__device__ __forceinline__ PagedBlock paged_block(const PagedArgs &a, int w, int lane) {
    const int G = a.H / a.H_kv;
    PagedBlock p{0, 0, 0, 0, 0, 0};
    if (a.cu_seqlens) {
        // sequence s owns the blocks from cu[s] G / 32 + s on, a few of which stay empty
        int lo = 0, hi = a.n_seq;
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const unsigned le = __ballot_sync(0xffffffffu, at < hi && min(max(a.cu_seqlens[at], 0), a.T) * G / kRows + at <= w);
            const int c = le == 0xffffffffu ? 32 : __ffs(~le) - 1;
            if (c == 0) break;
            hi = min(hi, lo + c * step);
            lo = lo + (c - 1) * step + 1;
        }
        p.s = lo - 1;
        if (p.s < 0) return p;
        p.c0 = min(max(a.cu_seqlens[p.s], 0), a.T);
        p.n = min(max(a.cu_seqlens[p.s + 1], p.c0), a.T) - p.c0;
        p.r0 = (w - p.c0 * G / kRows - p.s) * kRows;
    } else {
        const int each = (a.per_seq * G + kRows - 1) / kRows;
        p.s = w / each;
        p.c0 = p.s * a.per_seq;
        p.n = a.per_seq;
        p.r0 = (w - p.s * each) * kRows;
    }
    if (p.r0 >= p.n * G) {
        p.n = 0;
        return p;
    }
    const int L = a.cache_len ? min(max(a.cache_len[p.s], 0), a.max_len) : a.max_len;
    p.past = L - p.n;
    p.keys = max(0, p.past + min(p.r0 + kRows - 1, p.n * G - 1) / G + 1);
    return p;
}
// Keys of a split, in units of 8, at least 8 for each of the block's workers.
template <int W>
__device__ __forceinline__ int paged_share(int keys, int n_split) {
    return max(8 * W, ((keys + n_split - 1) / n_split + 7) / 8 * 8);
}

// Block x: (32 rows, cached head, split of the keys).  Up to eight splits are a cluster,
// whose first CTA writes the result; more leave their parts in the workspace.
template <int D, int W>
__global__ void __launch_bounds__(kThreads<W>, W == kMany<D> ? 1 : 2) paged_f32_kernel(const PagedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t f32_smem[];
    F32Smem<D, W> &sm = *reinterpret_cast<F32Smem<D, W> *>(f32_smem);
    const int tid = threadIdx.x, tx = tx_of(), G = a.H / a.H_kv;
    const bool cluster = a.n_split <= kTreeClusterF32;  // of a.n_split CTAs
    const int c = blockIdx.x % a.n_split, g = blockIdx.x / a.n_split % a.H_kv, w = blockIdx.x / a.n_split / a.H_kv;
    const PagedBlock p = paged_block(a, w, tid % 32);
    if (p.n == 0) return;  // as every CTA of the cluster
    const int rows = p.n * G, share = paged_share<W>(p.keys, a.n_split);
    const int k0 = static_cast<int>(min(static_cast<long long>(c) * share, static_cast<long long>(p.keys)));
    const int k1 = min(k0 + share, p.keys);
    if (k0 >= k1 && !cluster) return;  // the merge never reads this split
    for (int i = tid; i < kRows * D / 4; i += kThreads<W>) {
        const int r = p.r0 + i / (D / 4), col = 4 * (i % (D / 4));
        const bool in = r < rows;
        const float *q = static_cast<const float *>(a.q);
        if (in) q += static_cast<long long>(p.c0 + r / G) * a.q_ts + (g * G + r % G) * a.q_hs + col;
        cp_async16(smem_u32(&sm.q[i / (D / 4)][col]), q, in ? 16u : 0u);
    }
    cp_async_commit();
    int lim[4];  // rows see keys [0, lim)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = p.r0 + row_of(i);
        lim[i] = r < rows ? max(0, p.past + r / G + 1) : 0;
    }
    Rows4<D> st;
    reset(st);
    if (k0 < k1) {
        const int32_t *table = a.page_table + p.s * a.table_stride;
        struct Unit {
            const float *row;
            long long stride;
            bool in;
        };
        auto pages_at = [&](const float *base, long long ps, long long rs) {
            return [=](int key) {
                const int entry = page_of_key(a, key), page = table[entry];
                const bool in = is_page(a, page);  // an entry that is no page reads as zeros
                return Unit{base + (in ? page * ps + (key - entry * a.P) * rs : 0ll), rs, in};
            };
        };
        walk<D, W, true>(sm, pages_at(static_cast<const float *>(a.k) + g * a.k_hs, a.k_ps, a.k_rs),
                   pages_at(static_cast<const float *>(a.v) + g * a.v_hs, a.v_ps, a.v_rs), k0, k1, a.scale * kLog2e,
                   __any_sync(0xffffffffu, lim[0] > k0 || lim[1] > k0 || lim[2] > k0 || lim[3] > k0), st, [&](int i, int key0) {
                       uint32_t see = 0;
#pragma unroll
                       for (int j = 0; j < 4; ++j) see |= (key0 + tx + 8 * j < lim[i] ? 1u : 0u) << j;
                       return see;
                   }, rows - p.r0 <= 4);
    } else {
        cp_async_wait<0>();
    }
    Joined<D, W> x = join_workers(sm, st);
    if (cluster && !join_cluster(sm, x)) return;
    const int r = p.r0 + x.row();
    if (r >= rows) return;
    float *O;
    float f = 1.f;
    if (cluster) {
        const long long token = p.c0 + r / G;
        const int h = g * G + r % G;
        const bool live = p.past + r / G >= 0;
        O = static_cast<float *>(a.out) + token * a.o_ts + h * a.o_hs;
        f = 1.f / x.l;
        if (a.lse && x.column(0) == 0) a.lse[token * a.H + h] = live ? (x.m + log2f(x.l)) * kLn2 : -INFINITY;
        if (!live) {
#pragma unroll
            for (int cc = 0; cc < x.C; ++cc) x.o[cc] = make_float4(0.f, 0.f, 0.f, 0.f);
            f = 0.f;
        }
    } else {
        const size_t part = ((static_cast<size_t>(w) * a.H_kv + g) * kRows + x.row()) * a.n_split + c;
        O = a.part_o + part * D;
        if (x.column(0) == 0) *reinterpret_cast<float2 *>(a.part_ml + part * 2) = make_float2(x.m, x.l);
    }
#pragma unroll
    for (int cc = 0; cc < x.C; ++cc) *reinterpret_cast<float4 *>(O + x.column(cc)) = x.times(cc, f);
}

// One warp per row of a block: the parts of its splits.
template <int D, int W>
__global__ void __launch_bounds__(256) paged_merge_f32_kernel(const PagedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int G = a.H / a.H_kv, lane = threadIdx.x % 32, rr = blockIdx.x % (kRows / 8) * 8 + threadIdx.x / 32;
    const int g = blockIdx.x / (kRows / 8) % a.H_kv, w = blockIdx.x / (kRows / 8) / a.H_kv;
    const PagedBlock p = paged_block(a, w, lane);
    const int r = p.r0 + rr;
    if (p.n == 0 || r >= p.n * G || lane >= D / 4) return;
    const long long token = p.c0 + r / G;
    const int h = g * G + r % G, share = paged_share<W>(p.keys, a.n_split);
    const bool live = p.past + r / G >= 0;
    const size_t first = ((static_cast<size_t>(w) * a.H_kv + g) * kRows + rr) * a.n_split;
    float2 x[kAhead];
    float4 o[kAhead][1];
    const float2 ml = merge_row<1, false>(live ? (p.keys + share - 1) / share : 0, live,
                                          static_cast<float *>(a.out) + token * a.o_ts + h * a.o_hs + 4 * lane,
                                          [&](int c) { return reinterpret_cast<const float2 *>(a.part_ml)[first + c]; },
                                          [&](int c, int) { return reinterpret_cast<const float4 *>(a.part_o)[(first + c) * (D / 4) + lane]; },
                                          x, o);
    if (a.lse && lane == 0) a.lse[token * a.H + h] = live ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
}

template <int D, int W>
cudaError_t launch_paged_f32_w(const PagedArgs &a, unsigned blocks) {
    const size_t smem = sizeof(F32Smem<D, W>);
    cudaError_t e = cudaFuncSetAttribute(paged_f32_kernel<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const bool cluster = a.n_split <= kTreeClusterF32;
    e = launch_clusters(paged_f32_kernel<D, W>, cluster ? static_cast<unsigned>(a.n_split) : 1u, blocks * a.n_split,
                        kThreads<W>, smem, a.stream, a);
    if (e != cudaSuccess || cluster) return e;
    return launch_pdl(paged_merge_f32_kernel<D, W>, dim3(blocks * (kRows / 8)), dim3(256), 0, a.stream, a);
}

template <int D>
cudaError_t launch_paged_f32_t(const PagedArgs &a) {
    const unsigned blocks = static_cast<unsigned>(paged_f32_blocks(a) * a.H_kv);
    // More blocks than SMs: two an SM (as for trees).  Clusters of eight cannot take every
    // SM: of 16 with one block an SM one waits (eight sequences of 1000 keys, H 8 / 2: 16.5
    // against 10.5 us with two).
    const long long sms = a.n_split == 8 ? a.n_sm * 2 / 3 : a.n_sm;
    return blocks * static_cast<long long>(a.n_split) > sms ? launch_paged_f32_w<D, kMany<D> / 2>(a, blocks)
                                                            : launch_paged_f32_w<D, kMany<D>>(a, blocks);
}

}  // namespace

long long packed_f32_blocks(long long T, long long n_seq) { return T / kRows + n_seq; }

cudaError_t launch_packed_f32(const PackedArgs &a) {
    return a.D == 64 ? launch_packed_f32_t<64>(a) : launch_packed_f32_t<128>(a);
}

int tree_chunk_f32(int B, int H, int H_kv, int T, int Skv, int D, int n_sm) {
    // a few rounds of the blocks an SM holds, at least 128 keys a block (four sequences
    // of up to 1024 keys, splits merged by a second kernel: 14 us with 64 or 128 keys a
    // block, 18 with 256, 30 with 512; as a cluster of eight, 128 each: 12.4 us)
    const int rows = (H / H_kv) * T;
    const long long units = static_cast<long long>(B) * H_kv * ((rows + kRows - 1) / kRows);
    const long long tiles = (static_cast<long long>(Skv) + kKeys - 1) / kKeys;
    const long long want = 4LL * (n_sm > 0 ? n_sm : 1), least = 4;
    long long per = (units * tiles + want - 1) / want;
    per = (per + least - 1) / least * least;
    per = per < least ? least : per;
    per = per > tiles ? tiles : per;
    per = per < 1 ? 1 : per;
    return static_cast<int>(per * kKeys);
}

cudaError_t launch_tree_f32(const TreeArgs &a) {
    return a.D == 64 ? launch_tree_f32_t<64>(a) : launch_tree_f32_t<128>(a);
}

long long paged_f32_blocks(const PagedArgs &a) {
    const long long G = a.H / a.H_kv;
    return a.cu_seqlens ? a.T * G / kRows + a.n_seq : a.n_seq * ((a.per_seq * G + kRows - 1) / kRows);
}

int paged_f32_splits(const PagedArgs &a) {
    // Two blocks an SM (1 and 4: 43.3 and 44.1 against 39.1 us for 64 single tokens over 2000 keys, H 8 / 2,
    // D 64), 128 keys at least a block where the table's rows are full (64 and 256: 19.3 and
    // 16.9 against 11.7 us for four over 500 keys, H 32 / 8, D 128).
    const long long blocks = paged_f32_blocks(a) * a.H_kv, want = 2LL * (a.n_sm > 0 ? a.n_sm : 1);
    long long n = blocks > 0 ? want / blocks : 1;
    const long long most = (static_cast<long long>(a.max_len) + 127) / 128;
    n = n > most ? most : n;
    return static_cast<int>(n >= 2 * kTreeClusterF32 ? n : n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1);
}

cudaError_t launch_paged_f32(const PagedArgs &a) {
    return a.D == 64 ? launch_paged_f32_t<64>(a) : launch_paged_f32_t<128>(a);
}

}  // namespace attn
