// fp32 attention over tiles on the CUDA cores (FFMA only, no TF32): packed
// sequences (attn_fwd_packed) and trees of drafted tokens (attn_decode_tree).
//
// 32 query rows against tiles of 64 keys, online softmax in log2 units.  128
// threads hold the 32 x 64 scores as 4 x 4 each (rows 4 ty + i, keys tx + 16 j)
// and the 32 x D output as 4 rows x D / 16 columns each: a K or V element read
// from shared memory serves 4 rows, a Q or P element 4 keys or D / 16 columns, so
// the FMA pipe, not shared memory, is the bound.  The sixteen threads that
// share rows are half a warp: row sums are four shuffles, and P goes through
// shared memory without a block barrier.  K rows are padded by 16 bytes so that
// sixteen lanes read sixteen rows without conflicts.  The next tile's K is
// copied in (cp.async) while P V runs, its V while the scores are computed.
//
// Packed rows see keys [lo, hi) of the token axis.  A block's 32 rows may
// belong to several sequences: those are neighbours, so the block walks the
// keys from its first row's lo to its last row's hi and every row takes its own part.
// Tree rows see [0, hi) and the draft keys in their ancestor set.  A key that a
// row does not see contributes nothing whatever its row of V holds.
#include "kernels.h"
#include "ptx.cuh"
#include "serving.cuh"

#include <math.h>
#include <type_traits>

namespace attn {
namespace {

constexpr int kRows = 32;
constexpr int kKeys = 64;
constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct F32Smem {
    float q[kRows][D + 4];
    float k[kKeys][D + 4];
    float v[kKeys][D];
    float p[kRows][kKeys + 4];
    int lo[kRows], hi[kRows];
    Ancestors anc;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Running state of a thread's four rows.
template <int D>
struct Rows4 {
    float m[4], l[4];
    float o[4][D / 16];  // columns 64 c + 4 tx + e
};

// All tiles of keys [k0, k1): K row j at kbase + j * ks, V row j at vbase + j * vs.
// visible(i, key0) gives the bits of keys key0 + tx + 16 j, j < 4, of row 4 ty + i.
template <int D, typename Visible>
__device__ __forceinline__ void walk(F32Smem<D> &sm, const float *kbase, long long ks, const float *vbase, long long vs,
                                     int k0, int k1, float sl2, Rows4<D> &st, Visible visible) {
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    constexpr int C = D / 64;
    auto load = [&](float *dst, int stride, const float *base, long long gs, int key0) {
        const uint32_t to = smem_u32(dst);
        for (int i = tid; i < kKeys * D / 4; i += kThreads) {
            const int row = i / (D / 4), c = i % (D / 4);
            const bool in = key0 + row < k1;
            cp_async16(to + (row * stride + 4 * c) * 4, base + (in ? key0 + row : k0) * gs + 4 * c, in ? 16u : 0u);
        }
        cp_async_commit();
    };
    load(&sm.k[0][0], D + 4, kbase, ks, k0);
    load(&sm.v[0][0], D, vbase, vs, k0);
    for (int key0 = k0; key0 < k1; key0 += kKeys) {
        const bool more = key0 + kKeys < k1;
        cp_async_wait<1>();  // K of this tile (V may still be on its way)
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qa[4], kb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[i] = *reinterpret_cast<const float4 *>(&sm.q[4 * ty + i][d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) kb[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][d]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(qa[i].x, kb[j].x, s[i][j]);
                    s[i][j] = fmaf(qa[i].y, kb[j].y, s[i][j]);
                    s[i][j] = fmaf(qa[i].z, kb[j].z, s[i][j]);
                    s[i][j] = fmaf(qa[i].w, kb[j].w, s[i][j]);
                }
        }
        uint32_t hidden = 0;  // some row of the thread misses some key of the tile
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t see = visible(i, key0);
            hidden |= ~see & 15u;
            float mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = __fmul_rn(s[i][j], sl2);  // rounded before the difference below: huge scores
                if (see >> j & 1u) mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
            const float mn = fmaxf(st.m[i], mt);
            const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet (or nothing but -inf)
            const float corr = ex2_approx(st.m[i] - ref);
            st.m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = see >> j & 1u ? ex2_approx(s[i][j] - ref) : 0.f;
                sum += p;
                sm.p[4 * ty + i][tx + 16 * j] = p;
            }
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            st.l[i] = st.l[i] * corr + sum;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) st.o[i][e] *= corr;
        }
        // every row of the warp sees every key: plain FMAs; otherwise a weight
        // of zero must not meet an infinite or NaN value
        const bool edge = __any_sync(0xffffffffu, hidden != 0u);
        cp_async_wait<0>();  // V of this tile
        __syncthreads();     // all scores are done with K; P is visible
        if (more) load(&sm.k[0][0], D + 4, kbase, ks, key0 + kKeys);
        auto mix = [&](auto guarded) {
#pragma unroll 2
            for (int j = 0; j < kKeys; j += 4) {
                float4 p4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p4[i] = *reinterpret_cast<const float4 *>(&sm.p[4 * ty + i][j]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float4 x = *reinterpret_cast<const float4 *>(&sm.v[j + jj][64 * c + 4 * tx]);
                        const float xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = jj == 0 ? p4[i].x : jj == 1 ? p4[i].y : jj == 2 ? p4[i].z : p4[i].w;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y = fmaf(p, xv[e], st.o[i][4 * c + e]);
                                st.o[i][4 * c + e] = decltype(guarded)::value && p == 0.f ? st.o[i][4 * c + e] : y;
                            }
                        }
                    }
            }
        };
        if (edge)
            mix(std::true_type{});
        else
            mix(std::false_type{});
        __syncthreads();  // V and P are free
        if (more) load(&sm.v[0][0], D, vbase, vs, key0 + kKeys);
    }
    cp_async_wait<0>();
}

template <int D>
__device__ __forceinline__ void reset(Rows4<D> &st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        st.m[i] = -INFINITY;
        st.l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st.o[i][e] = 0.f;
    }
}

// ------------------------------------------------------------ packed sequences

template <int D>
__global__ void __launch_bounds__(kThreads) packed_f32_kernel(const PackedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t f32_smem[];
    F32Smem<D> &sm = *reinterpret_cast<F32Smem<D> *>(f32_smem);
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int h = blockIdx.y, g = h / (a.H / a.H_kv);
    const int t0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * kRows;
    for (int r = tid / 32; r < kRows; r += kThreads / 32) {
        const int t = t0 + r;
        const int s = min(count_le(a.cu_seqlens + 1, a.B, t, tid % 32), a.B - 1);
        if (tid % 32 == 0) {
            const int lo = min(max(a.cu_seqlens[s], 0), a.Sq), end = min(max(a.cu_seqlens[s + 1], lo), a.Sq);
            const bool live = t >= lo && t < end;
            sm.lo[r] = live ? lo : 0;
            sm.hi[r] = live ? (a.causal ? t + 1 : end) : 0;
        }
    }
    const float *Q = static_cast<const float *>(a.q) + h * a.q_hs;
    for (int i = tid; i < kRows * D / 4; i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + r < a.Sq) x = *reinterpret_cast<const float4 *>(Q + (t0 + r) * a.q_ts + 4 * c);
        *reinterpret_cast<float4 *>(&sm.q[r][4 * c]) = x;
    }
    __syncthreads();
    int k0 = 0x7fffffff, k1 = 0;
    for (int r = 0; r < kRows; ++r)
        if (sm.hi[r] > 0) {
            k0 = min(k0, sm.lo[r]);
            k1 = max(k1, sm.hi[r]);
        }
    if (k1 == 0) return;  // no token of a sequence here
    int lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = sm.lo[4 * ty + i];
        hi[i] = sm.hi[4 * ty + i];
    }
    Rows4<D> st;
    reset(st);
    walk<D>(sm, static_cast<const float *>(a.k) + g * a.k_hs, a.k_ts, static_cast<const float *>(a.v) + g * a.v_hs,
            a.v_ts, k0, k1, a.scale * kLog2e, st, [&](int i, int key0) {
                uint32_t see = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + tx + 16 * j;
                    see |= (key >= lo[i] && key < hi[i] ? 1u : 0u) << j;
                }
                return see;
            });
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (hi[i] == 0) continue;
        const long long t = t0 + 4 * ty + i;
        const float inv = 1.f / st.l[i];
        float *O = static_cast<float *>(a.out) + t * a.o_ts + h * a.o_hs;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<float4 *>(O + 64 * c + 4 * tx) = make_float4(
                st.o[i][4 * c] * inv, st.o[i][4 * c + 1] * inv, st.o[i][4 * c + 2] * inv, st.o[i][4 * c + 3] * inv);
        if (a.lse && tx == 0) a.lse[t * a.H + h] = (st.m[i] + log2f(st.l[i])) * kLn2;
    }
}

template <int D>
cudaError_t launch_packed_f32_t(const PackedArgs &a) {
    const size_t smem = sizeof(F32Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(packed_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.Sq + kRows - 1) / kRows), static_cast<unsigned>(a.H));
    return launch_pdl(packed_f32_kernel<D>, grid, dim3(kThreads), smem, a.stream, a);
}

// ------------------------------------------------------------ trees of drafted tokens

// Block x: (sequence and key/value head, split of the cache, 32 rows).
template <int D>
__global__ void __launch_bounds__(kThreads) tree_f32_kernel(const TreeArgs a, const int row_tiles) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) uint8_t f32_smem[];
    F32Smem<D> &sm = *reinterpret_cast<F32Smem<D> *>(f32_smem);
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int m = blockIdx.x % row_tiles, c = (blockIdx.x / row_tiles) % a.n_split;
    const int bk = blockIdx.x / row_tiles / a.n_split, b = bk / a.H_kv, g = bk % a.H_kv;
    const int G = a.H / a.H_kv, rows = G * a.T, r0 = m * kRows;
    const Draft d = draft_of(a, b);
    const int k0 = c * a.chunk, k1 = min(k0 + a.chunk, d.L);
    if (k0 >= k1 && a.n_split > 1) return;  // the merge never reads this split
    build_ancestors<kThreads>(a, b, d, sm.anc, tid, [] { __syncthreads(); });
    for (int i = tid; i < kRows * D / 4; i += kThreads) {
        const int r = r0 + i / (D / 4), col = 4 * (i % (D / 4));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && r % a.T < d.n)
            x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + b * a.q_bs +
                                                  (g * G + r / a.T) * a.q_hs + (r % a.T) * a.q_ts + col);
        *reinterpret_cast<float4 *>(&sm.q[i / (D / 4)][col]) = x;
    }
    bool live[4];
    const uint32_t *w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * ty + i, t = r % a.T;
        live[i] = r < rows && t < d.n && d.past + t >= 0;
        w[i] = sm.anc.bits[t];
    }
    Rows4<D> st;
    reset(st);
    const size_t head = static_cast<size_t>(bk) * a.Skv * D;
    if (k0 < k1) {
        __syncthreads();
        walk<D>(sm, static_cast<const float *>(a.k) + head, D, static_cast<const float *>(a.v) + head, D, k0, k1,
                a.scale * kLog2e, st, [&](int i, int key0) {
                    uint32_t see = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        see |= (visible32(w[i], key0 + 16 * j + tx - d.past) & 1u) << j;
                    return live[i] ? see : 0u;
                });
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * ty + i;
        if (r >= rows) continue;
        float *O;
        float f = 1.f;
        if (a.n_split == 1) {
            O = static_cast<float *>(a.out) + b * a.o_bs + (g * G + r / a.T) * a.o_hs + (r % a.T) * a.o_ts;
            f = live[i] ? 1.f / st.l[i] : 0.f;
        } else {
            const size_t part = (static_cast<size_t>(bk) * rows + r) * a.n_split + c;
            O = a.part_o + part * D;
            if (tx == 0) *reinterpret_cast<float2 *>(a.part_ml + part * 2) = make_float2(st.m[i], st.l[i]);
        }
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc)
            *reinterpret_cast<float4 *>(O + 64 * cc + 4 * tx) =
                make_float4(st.o[i][4 * cc] * f, st.o[i][4 * cc + 1] * f, st.o[i][4 * cc + 2] * f, st.o[i][4 * cc + 3] * f);
    }
}

template <int D>
cudaError_t launch_tree_f32_t(const TreeArgs &a) {
    const size_t smem = sizeof(F32Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(tree_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int row_tiles = ((a.H / a.H_kv) * a.T + kRows - 1) / kRows;
    const unsigned grid = static_cast<unsigned>(a.B * a.H_kv) * a.n_split * row_tiles;
    e = launch_pdl(tree_f32_kernel<D>, dim3(grid), dim3(kThreads), smem, a.stream, a, row_tiles);
    if (e != cudaSuccess || a.n_split == 1) return e;
    return launch_tree_merge_f32(a);
}

}  // namespace

cudaError_t launch_packed_f32(const PackedArgs &a) {
    return a.D == 64 ? launch_packed_f32_t<64>(a) : launch_packed_f32_t<128>(a);
}

cudaError_t launch_tree_f32(const TreeArgs &a) {
    return a.D == 64 ? launch_tree_f32_t<64>(a) : launch_tree_f32_t<128>(a);
}

}  // namespace attn
