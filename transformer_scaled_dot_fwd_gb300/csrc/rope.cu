// Rotary positions, and their append to a KV cache, in one pass over the rows.
//
// A head row of D elements holds r / 2 pairs, (x[p], x[p + r/2]) in the half
// layout or (x[2p], x[2p + 1]) in the interleaved one; elements from r on stay
// as they are.  Pair p of a token at position n is turned by the angle n w_p:
//     (a, b) -> mscale (a cos - b sin, b cos + a sin),
// with sin negated for the inverse turn (mscale R(-n), which is also the
// gradient of the turn).  The turn keeps q_m . k_n a function of m - n.
//
// Angles.  n w_p reaches 10^5 .. 10^9 radians for far positions, where a
// 32-bit product has lost every digit of the angle.  w_p / 2 pi is held as a
// 64-bit fixed-point fraction of a turn, so n times it modulo 2^64 is the exact
// fraction of a turn left over (one 64-bit multiply, wrapping included, and
// the right one for negative n too); its top 32 bits go to sincospif.
//
// The rows are read once and written once: bound by HBM for prompts, by the
// launch and one round trip for a step of single tokens.  A block takes one or two
// tokens with all their heads: the r / 2 angles of a token are computed once
// into shared memory and serve every head of q and k.  Small blocks of 128
// threads, many to an SM, hide one block's look-ups behind another's rows: 256
// threads and 8 tokens a block took 74 us instead of 68 for 16385 tokens of
// 32 + 8 heads into a cache, and several units in flight per thread, at the price
// of fewer blocks, 100 us and more.  A thread then handles
// units of VEC pairs: two 16-byte loads, 2 VEC elements turned in fp32 and
// rounded once, two 16-byte stores.  Rows whose strides, addresses or rotary
// depth do not allow 16-byte accesses take the same code with VEC = 1.
#include "kernels.h"
#include "ptx.cuh"
#include "serving.cuh"

namespace attn {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float *y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 *y) { *y = __float2bfloat16_rn(x); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T x[VEC];
};

struct Token {
    long long cache_row;  // (b * H_kv) * Skv + row of head 0's cache row, or -1: not cached
    int position;
    int live;             // 0: the token belongs to no sequence and stays untouched
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, const int tokens, const int rows_per_block) {
    __shared__ float2 turn[kRopeMaxTokens][64];
    __shared__ Token tok[kRopeMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, a.T - t0);
    const bool append = a.kcache != nullptr;

    for (int i = warp; i < nt; i += kRopeWarps) {
        const int t = t0 + i;
        Token k{-1, 0, 1};
        if (append) {
            int b, n, at;  // sequence, its tokens, this token's index
            if (a.cu_seqlens) {
                b = count_le(a.cu_seqlens + 1, a.B, t, lane);
                const int first = a.cu_seqlens[min(b, a.B - 1)];
                n = a.cu_seqlens[min(b, a.B - 1) + 1] - first;
                at = t - first;
                k.live = b < a.B && at >= 0 && at < n;
            } else {
                n = a.T / a.B;
                b = t / n;
                at = t - b * n;
            }
            if (k.live) {
                const int L = a.cache_len ? min(max(a.cache_len[b], 0), a.Skv) : a.Skv;
                const int row = L - n + at;  // 0 <= at < n and L >= 0: no overflow
                k.position = row;
                if (row >= 0) k.cache_row = static_cast<long long>(b) * a.H_kv * a.Skv + row;
            }
        }
        if (a.positions) k.position = a.positions[t];
        if (lane == 0) tok[i] = k;
    }
    __syncthreads();
    const int half = a.rotary_dim / 2;
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int k = i / half, p = i - k * half;
        // fraction of a turn, as half turns in [-1, 1): sincospif takes those
        const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(tok[k].position)) * a.turns[p];
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 0x1p-31f, &s, &c);
        turn[k][p] = make_float2(c * a.mscale, s * a.sin_scale);
    }
    __syncthreads();

    constexpr int U64 = 64 / (2 * VEC);  // units of 64 elements
    const int units = a.D == 128 ? 2 * U64 : U64;
    const int ushift = 31 - __clz(units);  // a power of two
    const int r0 = blockIdx.y * rows_per_block;
    const int rows = min(rows_per_block, a.H + a.H_kv * (append ? 2 : 1) - r0);
    const int turned_units = half / VEC;

    for (int i = threadIdx.x; i < (nt * rows) << ushift; i += kRopeThreads) {
        const int u = i & (units - 1);
        const int k = (i >> ushift) / rows;
        const int r = r0 + (i >> ushift) - k * rows;
        if (!tok[k].live) continue;
        const size_t t = static_cast<size_t>(t0 + k);
        const T *src;
        T *dst = nullptr, *cache = nullptr;
        bool turned = u < turned_units;
        if (r < a.H) {
            src = static_cast<const T *>(a.q) + t * a.q_ts + r * a.q_hs;
            dst = static_cast<T *>(a.q_out) + t * a.qo_ts + r * a.qo_hs;
        } else {
            const bool is_v = r >= a.H + a.H_kv;
            const int g = r - a.H - (is_v ? a.H_kv : 0);
            if (is_v) {
                src = static_cast<const T *>(a.v) + t * a.v_ts + g * a.v_hs;
                turned = false;
            } else {
                src = static_cast<const T *>(a.k) + t * a.k_ts + g * a.k_hs;
                if (a.k_out) dst = static_cast<T *>(a.k_out) + t * a.ko_ts + g * a.ko_hs;
            }
            if (append && tok[k].cache_row >= 0)
                cache = static_cast<T *>(is_v ? a.vcache : a.kcache) +
                        (tok[k].cache_row + static_cast<long long>(g) * a.Skv) * a.D;
        }
        if (!turned && dst == src) dst = nullptr;  // in place: nothing to copy
        if (!dst && !cache) continue;
        const int e0 = turned && !a.interleaved ? u * VEC : 2 * u * VEC;
        const int e1 = turned && !a.interleaved ? half + u * VEC : e0 + VEC;
        using V = Vec<T, VEC>;
        V x = *reinterpret_cast<const V *>(src + e0), y = *reinterpret_cast<const V *>(src + e1);
        if (turned) {
            const float2 *cs = &turn[k][u * VEC];
            if (a.interleaved) {
                // element 2 VEC u + e of the unit: pairs sit side by side
                V z[2] = {x, y};
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    T &pa = z[(2 * e) / VEC].x[(2 * e) % VEC], &pb = z[(2 * e + 1) / VEC].x[(2 * e + 1) % VEC];
                    const float va = to_f32(pa), vb = to_f32(pb);
                    from_f32(va * cs[e].x - vb * cs[e].y, &pa);
                    from_f32(vb * cs[e].x + va * cs[e].y, &pb);
                }
                x = z[0];
                y = z[1];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float va = to_f32(x.x[e]), vb = to_f32(y.x[e]);
                    from_f32(va * cs[e].x - vb * cs[e].y, &x.x[e]);
                    from_f32(vb * cs[e].x + va * cs[e].y, &y.x[e]);
                }
            }
        }
        if (dst) {
            *reinterpret_cast<V *>(dst + e0) = x;
            *reinterpret_cast<V *>(dst + e1) = y;
        }
        if (cache) {
            *reinterpret_cast<V *>(cache + e0) = x;
            *reinterpret_cast<V *>(cache + e1) = y;
        }
    }
}

template <typename T, int VEC>
cudaError_t launch_rope_t(const RopeArgs &a) {
    const int rows = a.H + a.H_kv * (a.kcache ? 2 : 1);
    const long long sms = a.n_sm > 0 ? a.n_sm : 1;
    // two tokens a block when that still leaves several rounds of blocks an SM;
    // with few tokens the rows of one are split
    int tokens = kRopeMaxTokens;
    while (tokens > 1 && (a.T + tokens - 1) / tokens < 32 * sms) tokens /= 2;
    const long long blocks = (a.T + tokens - 1) / tokens;
    const int units = rows * (a.D / (2 * VEC));
    long long split = (2 * sms + blocks - 1) / blocks;
    const long long most = (units + kRopeThreads - 1) / kRopeThreads;
    split = split > most ? most : split;
    const int per = static_cast<int>((rows + split - 1) / split);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((rows + per - 1) / per));
    return launch_pdl(rope_kernel<T, VEC>, grid, dim3(kRopeThreads), 0, a.stream, a, tokens, per);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool f32, bool wide) {
    if (f32) return wide ? launch_rope_t<float, 4>(a) : launch_rope_t<float, 1>(a);
    return wide ? launch_rope_t<__nv_bfloat16, 8>(a) : launch_rope_t<__nv_bfloat16, 1>(a);
}

}  // namespace attn
