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
// 64-bit fixed-point fraction of a turn, right to its last unit (rope_turns.h), so n
// times it modulo 2^64 is the fraction of a turn left over, off by |n| units, 2^-33 of
// a turn at most (one 64-bit multiply, wrapping included, and the right one for
// negative n too); its top 32 bits go to sincospif as a float.
//
// The rows are read once and written once: bound by HBM for prompts, by the
// launch and one round trip for a step of single tokens.  A block takes one or two
// tokens with all their heads; the r / 2 angles of a token are computed once.  A
// thread keeps one unit of VEC pairs of every few rows, its cosines and sines in
// registers: two 16-byte loads, 2 VEC elements turned in fp32 and rounded once,
// two 16-byte stores a row.  Rows whose strides, addresses or rotary depth do not
// allow 16-byte accesses take the same code with VEC = 1.
//
// Small blocks, ten and more to an SM, hide one block's look-ups behind another's
// rows.  16385 tokens of 32 + 8 heads of depth 128 into a cache (402 MB moved): 66
// us, 6.1 TB/s; 256 threads and 8 tokens a block took 74 us, two rows in flight
// per thread at 106 registers 109 us.  32768 tokens of 64 heads, half of each
// turned (1.07 GB): 164 us, 6.5 TB/s.  A step of 64 tokens into a cache: 3.2 us.  With a
// rotary depth of 36 (VEC = 1, single elements) the first takes 211 us, the second 505.
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

// VEC elements, as the 16 bytes (or the single element) they are moved in.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Vec {
    T x[VEC];
};
template <>
struct alignas(16) Vec<__nv_bfloat16, 8> {
    uint32_t w[4];  // two elements each
};

// (a, b) -> (a c - b s, b c + a s), a and b the elements of x and of y.
template <typename T, int VEC>
__device__ __forceinline__ void turn_halves(Vec<T, VEC> &x, Vec<T, VEC> &y, const Vec<float, VEC> &c,
                                            const Vec<float, VEC> &s) {
#pragma unroll
    for (int p = 0; p < VEC; ++p) {
        const float a = to_f32(x.x[p]), b = to_f32(y.x[p]);
        from_f32(a * c.x[p] - b * s.x[p], &x.x[p]);
        from_f32(b * c.x[p] + a * s.x[p], &y.x[p]);
    }
}
__device__ __forceinline__ void turn_halves(Vec<__nv_bfloat16, 8> &x, Vec<__nv_bfloat16, 8> &y, const Vec<float, 8> &c,
                                            const Vec<float, 8> &s) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float a0 = bf16lo_to_f32(x.w[p]), a1 = bf16hi_to_f32(x.w[p]);
        const float b0 = bf16lo_to_f32(y.w[p]), b1 = bf16hi_to_f32(y.w[p]);
        x.w[p] = pack_bf16x2(a0 * c.x[2 * p] - b0 * s.x[2 * p], a1 * c.x[2 * p + 1] - b1 * s.x[2 * p + 1]);
        y.w[p] = pack_bf16x2(b0 * c.x[2 * p] + a0 * s.x[2 * p], b1 * c.x[2 * p + 1] + a1 * s.x[2 * p + 1]);
    }
}
// The same for pairs that sit side by side in the 2 VEC elements of x and y.
template <typename T, int VEC>
__device__ __forceinline__ void turn_side_by_side(Vec<T, VEC> &x, Vec<T, VEC> &y, const Vec<float, VEC> &c,
                                                  const Vec<float, VEC> &s) {
    T z[2 * VEC];
#pragma unroll
    for (int p = 0; p < VEC; ++p) z[p] = x.x[p], z[VEC + p] = y.x[p];
#pragma unroll
    for (int p = 0; p < VEC; ++p) {
        const float a = to_f32(z[2 * p]), b = to_f32(z[2 * p + 1]);
        from_f32(a * c.x[p] - b * s.x[p], &z[2 * p]);
        from_f32(b * c.x[p] + a * s.x[p], &z[2 * p + 1]);
    }
#pragma unroll
    for (int p = 0; p < VEC; ++p) x.x[p] = z[p], y.x[p] = z[VEC + p];
}
__device__ __forceinline__ void turn_side_by_side(Vec<__nv_bfloat16, 8> &x, Vec<__nv_bfloat16, 8> &y,
                                                  const Vec<float, 8> &c, const Vec<float, 8> &s) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        uint32_t &w = p < 4 ? x.w[p] : y.w[p - 4];
        const float a = bf16lo_to_f32(w), b = bf16hi_to_f32(w);
        w = pack_bf16x2(a * c.x[p] - b * s.x[p], b * c.x[p] + a * s.x[p]);
    }
}

struct Token {
    long long cache_row;  // (b * H_kv) * Skv + row of head 0's cache row, or -1: not cached
    int position;
    int live;             // 0: the token belongs to no sequence and stays untouched
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kRopeThreads, 10)
    rope_kernel(const __grid_constant__ RopeArgs a, const int tokens, const int rows_per_block) {
    __shared__ __align__(16) float cosines[kRopeMaxTokens][64], sines[kRopeMaxTokens][64];
    __shared__ Token tok[kRopeMaxTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, a.T - t0);
    const bool append = a.append != 0;

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
        cosines[k][p] = c * a.mscale;
        sines[k][p] = s * a.sin_scale;
    }
    __syncthreads();

    constexpr int U64 = 64 / (2 * VEC);  // units of 64 elements
    const int units = a.D == 128 ? 2 * U64 : U64;
    const int ushift = 31 - __clz(units);  // a power of two
    const int r0 = blockIdx.y * rows_per_block;
    const int rows = min(rows_per_block, a.H + a.H_kv * (append ? 2 : 1) - r0);
    // A thread keeps one unit of every step-th row, so the angles of a token stay in
    // registers over its rows.
    const int u = threadIdx.x & (units - 1), step = kRopeThreads >> ushift;
    using V = Vec<T, VEC>;
    for (int k = 0; k < nt; ++k) {
        const Token token = tok[k];
        if (!token.live) continue;
        const size_t t = static_cast<size_t>(t0 + k);
        Vec<float, VEC> c, s;
        if (u < half / VEC) {
            c = *reinterpret_cast<const Vec<float, VEC> *>(&cosines[k][u * VEC]);
            s = *reinterpret_cast<const Vec<float, VEC> *>(&sines[k][u * VEC]);
        }
        for (int r = r0 + (threadIdx.x >> ushift); r < r0 + rows; r += step) {
            const T *src;
            T *dst = nullptr, *cache = nullptr;
            bool turned = u < half / VEC;
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
                if (append && token.cache_row >= 0)
                    cache = static_cast<T *>(is_v ? a.vcache : a.kcache) +
                            (token.cache_row + static_cast<long long>(g) * a.Skv) * a.D;
            }
            if (!turned && dst == src) dst = nullptr;  // in place: nothing to copy
            if (!dst && !cache) continue;
            const int e0 = turned && !a.interleaved ? u * VEC : 2 * u * VEC;
            const int e1 = turned && !a.interleaved ? half + u * VEC : e0 + VEC;
            V x = *reinterpret_cast<const V *>(src + e0), y = *reinterpret_cast<const V *>(src + e1);
            if (turned) {
                if (a.interleaved)
                    turn_side_by_side(x, y, c, s);
                else
                    turn_halves(x, y, c, s);
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
}

template <typename T, int VEC>
cudaError_t launch_rope_t(const RopeArgs &a) {
    const int rows = a.H + a.H_kv * (a.append ? 2 : 1);
    const long long sms = a.n_sm > 0 ? a.n_sm : 1;
    // two tokens a block when that still leaves several rounds of blocks an SM;
    // with few tokens the rows of one are split
    int tokens = kRopeMaxTokens;
    while (tokens > 1 && a.T / tokens < 32 * sms) tokens /= 2;
    const long long blocks = (static_cast<long long>(a.T) + tokens - 1) / tokens;
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
