// Device helpers shared by the packed, rotary and tree kernels: the sequence of
// a token, what a drafted token sees of its tree, merges of partial results.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

#include <type_traits>

namespace attn {

// Number of the n nondecreasing values v[0..n) that are <= t, found by the
// whole warp with 32 probes a step.  Any contents of v end the search.
__device__ __forceinline__ int count_le(const int32_t *v, int n, int t, int lane) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, at < hi && v[at] <= t);
        const int c = le == 0xffffffffu ? 32 : __ffs(~le) - 1;  // leading probes that hold
        if (c == 0) break;
        hi = min(hi, lo + c * step);
        lo = lo + (c - 1) * step + 1;
    }
    return lo;
}

// What the draft of one sequence looks like: L cache rows, the last n of them
// drafted, so draft token j's key sits at row past + j (none when negative).
struct Draft {
    int L, n, past;
};

__device__ __forceinline__ Draft draft_of(const TreeArgs &a, int b) {
    Draft d;
    d.L = a.cache_len ? min(max(a.cache_len[b], 0), a.Skv) : a.Skv;
    d.n = a.draft_len ? min(max(a.draft_len[b], 0), a.T) : a.T;
    d.past = d.L - d.n;
    return d;
}

// Bit sets of each drafted token's visible draft keys: itself and its
// ancestors, as far as they have a cache row.  `Threads` threads call it
// together, `sync` joins them.  The parent relation is closed by doubling: after
// round i a set holds the 2^i nearest ancestors.
struct alignas(16) Ancestors {
    uint32_t bits[kTreeMaxTokens][4];
    int jump[kTreeMaxTokens];
};

template <int Threads, typename Sync>
__device__ __forceinline__ void build_ancestors(const TreeArgs &a, int b, const Draft &d, Ancestors &anc, int tid,
                                                Sync sync) {
    constexpr int kEach = kTreeMaxTokens / Threads;  // tokens tid, tid + Threads, ...
    int jump[kEach];
    uint32_t w[kEach][4];
#pragma unroll
    for (int y = 0; y < kEach; ++y) {
        const int t = tid + y * Threads;
        jump[y] = -1;
        if (t < d.n) {
            const int p = a.parents[b * a.parents_bs + t];
            jump[y] = p >= 0 && p < t ? p : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[y][i] = t < d.n && d.past + t >= 0 && t / 32 == i ? 1u << (t % 32) : 0u;
            anc.bits[t][i] = w[y][i];
        }
        anc.jump[t] = jump[y];
    }
    sync();
    for (int reach = 1; reach < d.n; reach *= 2) {
        int next[kEach];
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            next[y] = -1;
            if (jump[y] >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[y][i] |= anc.bits[jump[y]][i];
                next[y] = anc.jump[jump[y]];
                if (next[y] >= jump[y]) next[y] = -1;  // never, unless a wait gave up: stay inside the set
            }
        }
        sync();
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            const int t = tid + y * Threads;
            if (jump[y] >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) anc.bits[t][i] = w[y][i];
                anc.jump[t] = jump[y] = next[y];
            }
        }
        sync();
    }
}

// Visibility of draft-relative keys [s, s + 32) for a token with ancestor
// words w: keys before 0 are the committed cache, keys from 128 on nothing.
__device__ __forceinline__ uint32_t visible32(const uint32_t *w, int s) {
    if (s <= -32) return 0xffffffffu;
    if (s >= kTreeMaxTokens) return 0u;
    if (s < 0) return ((1u << -s) - 1u) | (w[0] << -s);
    const int i = s / 32, r = s % 32;
    const uint32_t lo = w[i], hi = i < 3 ? w[i + 1] : 0u;
    return __funnelshift_r(lo, hi, r);
}

// Any bf16 of the pair w infinite or NaN (exponent bits all ones)?
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); }

// Clean the V tile at shared address `tile` (kSub blocks of kRows rows of 128
// bytes; kGroups: kRows / 8 groups of kSub blocks of 8 rows) for an MMA: rows from
// `inside` on become zeros, non-finite elements of the others too.  Returns whether this thread met one.  `Threads` threads share
// the tile.  An exponent of all ones carries into the sign bit when one is added
// to it, so three operations test a pair of bf16, and eight 16-byte loads are in
// flight before the first test.
template <int kSub, int kRows, int Threads, bool kGroups = false>
__device__ __forceinline__ bool clean_v_tile(uint32_t tile, int inside, int tid) {
    constexpr int kChunks = kSub * kRows * 8, kBatch = 8;
    static_assert(kChunks % (Threads * kBatch) == 0, "whole batches");
    bool bad = false;
    // row of 16-byte chunk c
    auto row_of = [](int c) { return kGroups ? (c / (kSub * 64)) * 8 + (c >> 3) % 8 : (c >> 3) % kRows; };
    auto pass = [&](auto partial) {
#pragma unroll 1
        for (int c0 = tid; c0 < kChunks; c0 += Threads * kBatch) {
            uint4 v[kBatch];
            uint32_t acc = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = ld_shared_v4(tile + (c0 + i * Threads) * 16);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (decltype(partial)::value && row_of(c0 + i * Threads) >= inside) {
                    st_shared_v4(tile + (c0 + i * Threads) * 16, 0u, 0u, 0u, 0u);
                    continue;
                }
                acc |= ((v[i].x & 0x7f807f80u) + 0x00800080u) | ((v[i].y & 0x7f807f80u) + 0x00800080u) |
                       ((v[i].z & 0x7f807f80u) + 0x00800080u) | ((v[i].w & 0x7f807f80u) + 0x00800080u);
            }
            if (!(acc & 0x80008000u)) continue;
            // read again, one chunk at a time: nothing stays live for a rare case
#pragma unroll 1
            for (int c = c0; c < c0 + kBatch * Threads; c += Threads) {
                if (decltype(partial)::value && row_of(c) >= inside) continue;
                const uint4 v = ld_shared_v4(tile + c * 16);
                const uint32_t n0 = nonfinite2(v.x), n1 = nonfinite2(v.y), n2 = nonfinite2(v.z), n3 = nonfinite2(v.w);
                if (n0 | n1 | n2 | n3) {
                    bad = true;
                    st_shared_v4(tile + c * 16, v.x & ~n0, v.y & ~n1, v.z & ~n2, v.w & ~n3);
                }
            }
        }
    };
    if (inside >= kRows)
        pass(std::false_type{});
    else
        pass(std::true_type{});
    return bad;
}

// ------------------------------------------------------------ merges of partial results

__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c, M the largest m_c, the
// parts added in order, for one row and 4 C columns: part(c) is the row's (m, l) in
// part c, column(c, e) its e-th four columns.
//
// kAhead parts are loaded before the first is used: few rows, so latency counts.  Early:
// x and o hold the first ones already.  Returns (M, sum).
constexpr int kAhead = 4;
template <int C, bool Early, typename T, typename Part, typename Column>
__device__ __forceinline__ float2 merge_row(int n, bool live, T *out, Part part, Column column,
                                          float2 (&x)[kAhead], float4 (&o)[kAhead][C]) {
    float4 acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, M = -INFINITY;
    auto add = [&](int c0) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            if (c0 + y >= n) break;
            // relative to the running max; a part in which the row saw nothing holds zeros
            const float mn = fmaxf(M, x[y].x), ref = mn == -INFINITY ? 0.f : mn;
            const float old = ex2_approx(M - ref), w = ex2_approx(x[y].x - ref);
            M = mn;
            sum = sum * old + w * x[y].y;
#pragma unroll
            for (int e = 0; e < C; ++e)
                acc[e] = make_float4(fmaf(w, o[y][e].x, acc[e].x * old), fmaf(w, o[y][e].y, acc[e].y * old),
                                     fmaf(w, o[y][e].z, acc[e].z * old), fmaf(w, o[y][e].w, acc[e].w * old));
        }
    };
    auto load = [&](int c0) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int c = min(c0 + y, n - 1);
            x[y] = part(c);
#pragma unroll
            for (int e = 0; e < C; ++e) o[y][e] = column(c, e);
        }
    };
    for (int c0 = 0; c0 < n; c0 += kAhead) {
        if (!Early || c0 > 0) load(c0);
        add(c0);
    }
    const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < C; ++e)
        store4(out + 4 * e, live ? make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv)
                                 : make_float4(0.f, 0.f, 0.f, 0.f));
    return make_float2(M, sum);
}

}  // namespace attn
