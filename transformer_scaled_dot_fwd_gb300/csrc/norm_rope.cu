// RMS norm of each head row of q and k, the rotary turn, and the append of keys and
// values to the pages of a cache, in one pass over the rows.
//
//     y = x / sqrt(mean(x^2) + eps) * w,   then pairs of y turned by n w_p (rope.cu),
// in fp32 from the load to the one rounding at the store; a tensor without weights is
// turned as it is.  What each turned row costs beside its read and write is one sum over
// D / (2 VEC) neighbouring lanes, three or four shuffles in the wide form.
//
// The rows are read once and written once (the append writes k and v to their pages
// instead): bound by HBM for prompts, by the launch and two dependent look-ups (sequence,
// page) for a step of single tokens.  As in rope.cu a block takes one or two tokens with
// all their heads and computes a token's angles once.  A thread keeps one unit of VEC pairs
// of every few rows and loads one row ahead, the first one before the look-ups, whose two
// or three round trips would otherwise stand in front of every block's rows; angles and
// weights are read again with each row, from shared memory and L1.
//
// The arithmetic of a row is most of the issue slots (some 200 instructions for 4 rows
// of a warp), so it goes two elements at a time (f32x2), each value with the roundings that
// rope.cu's turn has, and the layouts of the pairs are two kernels.
//
// Measured: 16385 tokens of 32 + 8 heads of depth 128 into pages of 64 rows (402 MB moved)
// 68.5 us, 5.9 TB/s; a step of 64 tokens 4.9 us a call, 3.5 of them in the kernel.  Eight
// blocks an SM 70.6 us, ten 72.5 (registers spill); element by element 74; both layouts in
// one kernel 2 us more; two or three rows ahead 78-89 us (fewer blocks an SM); without
// the load ahead 82-89 us.  One token a block 80 us, three to eight as two.
//
// Rows whose addresses, strides or pairs do not allow 16-byte accesses take VEC = 1, with
// a warp a row.  Interleaved pairs need no multiple of VEC: the unit in which the turned
// ones end chooses pair by pair.
#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"
#include "serving.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kResident = 9;  // blocks an SM: 56 registers a thread
constexpr int kTokens = 2;  // a block takes at most

// VEC elements, as the 16 bytes (or the single element) they are moved in.
template <typename T, int VEC>
struct Unit;
template <>
struct Unit<float, 4> {
    float4 v;
    __device__ __forceinline__ void unpack(float *x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
    __device__ __forceinline__ void pack(const float *x) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Unit<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void unpack(float *x) const {
        x[0] = bf16lo_to_f32(v.x), x[1] = bf16hi_to_f32(v.x), x[2] = bf16lo_to_f32(v.y), x[3] = bf16hi_to_f32(v.y);
        x[4] = bf16lo_to_f32(v.z), x[5] = bf16hi_to_f32(v.z), x[6] = bf16lo_to_f32(v.w), x[7] = bf16hi_to_f32(v.w);
    }
    __device__ __forceinline__ void pack(const float *x) {
        v = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Unit<float, 1> {
    float v;
    __device__ __forceinline__ void unpack(float *x) const { x[0] = v; }
    __device__ __forceinline__ void pack(const float *x) { v = x[0]; }
};
template <>
struct Unit<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void unpack(float *x) const { x[0] = __bfloat162float(v); }
    __device__ __forceinline__ void pack(const float *x) { v = __float2bfloat16_rn(x[0]); }
};

struct Token {
    long long k_at, v_at;  // elements from the pools' start to the token's row of head 0
    int position;
    int live;              // 0: the token belongs to no sequence and stays untouched
    int cached;            // the token has a page
};

template <typename T, int VEC, int D, bool Interleaved>
__global__ void __launch_bounds__(kThreads, kResident)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const int tokens, const int rows_per_block) {
    constexpr int kUnits = D / (2 * VEC);                // of a row
    constexpr int kLanes = kUnits < 32 ? kUnits : 32;    // that share a row
    constexpr int kEach = kUnits / kLanes;               // units of a lane
    constexpr int kGroups = kThreads / kLanes;
    using U = Unit<T, VEC>;
    __shared__ __align__(16) float cosines[kTokens][64], sines[kTokens][64];
    __shared__ Token tok[kTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, a.T - t0);
    const bool append = a.append != 0;
    const bool interleaved = VEC > 1 ? Interleaved : a.interleaved != 0;
    const int half = a.rotary_dim / 2;
    const int u0 = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int r0 = blockIdx.y * rows_per_block;
    const int r1 = min(r0 + rows_per_block, a.H + a.H_kv * (append ? 2 : 1));

    // A thread's rows, token by token, one loaded ahead of the one at work; the first
    // loads are on their way during the look-ups.
    struct Place {
        int k, r;  // token of the block, row
    };
    auto next = [&](Place &p) {
        p.r += kGroups;
        if (p.r >= r1) p.r = r0 + group, ++p.k;
    };
    auto columns = [&](int r, int y, int *e0, int *e1) {
        const int u = u0 + y * kLanes;
        const bool split = r < a.H + a.H_kv && !interleaved && u * VEC < half;  // the pairs' second halves lie apart
        *e0 = split ? u * VEC : 2 * u * VEC;
        *e1 = split ? half + u * VEC : 2 * u * VEC + VEC;
    };
    auto load = [&](const Place &p, U *lo, U *hi) {
        if (p.k >= nt || p.r >= r1) return;
        const size_t t = static_cast<size_t>(t0 + p.k);
        const T *src;
        if (p.r < a.H)
            src = static_cast<const T *>(a.q) + t * a.q_ts + p.r * a.q_hs;
        else if (p.r < a.H + a.H_kv)
            src = static_cast<const T *>(a.k) + t * a.k_ts + (p.r - a.H) * a.kt_hs;
        else
            src = static_cast<const T *>(a.v) + t * a.v_ts + (p.r - a.H - a.H_kv) * a.vt_hs;
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            int e0, e1;
            columns(p.r, y, &e0, &e1);
            lo[y] = *reinterpret_cast<const U *>(src + e0);
            hi[y] = *reinterpret_cast<const U *>(src + e1);
        }
    };
    Place at{0, r0 + group};
    U lo[kEach], hi[kEach];
    load(at, lo, hi);

    for (int i = warp; i < nt; i += kWarps) {
        const int t = t0 + i;
        Token k{0, 0, 0, 1, 0};
        if (append) {
            int b, n, index;  // sequence, its tokens, this token's index
            if (a.cu_seqlens) {
                b = count_le(a.cu_seqlens + 1, a.n_seq, t, lane);
                const int first = a.cu_seqlens[min(b, a.n_seq - 1)];
                n = a.cu_seqlens[min(b, a.n_seq - 1) + 1] - first;
                index = t - first;
                k.live = b < a.n_seq && index >= 0 && index < n;
            } else {
                n = a.T / a.n_seq;
                b = t / n;
                index = t - b * n;
            }
            if (k.live) {
                const int L = a.cache_len ? min(max(a.cache_len[b], 0), a.max_len) : a.max_len;
                const int row = L - n + index;  // 0 <= index < n and L >= 0: no overflow
                k.position = row;
                if (row >= 0) {
                    const int page = a.page_table[b * a.table_stride + row / a.P];
                    k.cached = page >= 0 && page < a.n_pages;
                    k.k_at = page * a.k_ps + row % a.P * a.k_rs;
                    k.v_at = page * a.v_ps + row % a.P * a.v_rs;
                }
            }
        }
        if (a.positions) k.position = a.positions[t];
        if (lane == 0) tok[i] = k;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int k = i / half, p = i - k * half;
        // fraction of a turn, as half turns in [-1, 1): sincospif takes those
        const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(tok[k].position)) * a.turns[p];
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 0x1p-31f, &s, &c);
        cosines[k][p] = c * a.mscale;
        sines[k][p] = s * a.mscale;
    }
    __syncthreads();

    const unsigned mask = kLanes == 32 ? 0xffffffffu : ((1u << (kLanes & 31)) - 1u) << (lane - lane % kLanes);
    while (at.k < nt && at.r < r1) {
        const Place now = at;
        U x_lo[kEach], x_hi[kEach];
#pragma unroll
        for (int y = 0; y < kEach; ++y) x_lo[y] = lo[y], x_hi[y] = hi[y];
        next(at);
        load(at, lo, hi);
        const int r = now.r;
        const long long t = t0 + now.k;
        if (!tok[now.k].live) continue;
        const bool cached = tok[now.k].cached, is_v = r >= a.H + a.H_kv;
        const T *w = nullptr;
        T *dst = nullptr, *cache = nullptr;
        if (r < a.H) {
            dst = static_cast<T *>(a.q_out) + t * a.qo_ts + r * a.qo_hs;
            w = static_cast<const T *>(a.q_weight);
        } else if (!is_v) {
            const int g = r - a.H;
            if (a.k_out) dst = static_cast<T *>(a.k_out) + t * a.ko_ts + g * a.ko_hs;
            if (cached) cache = static_cast<T *>(a.kpages) + tok[now.k].k_at + g * a.k_hs;
            w = static_cast<const T *>(a.k_weight);
        } else if (cached) {
            cache = static_cast<T *>(a.vpages) + tok[now.k].v_at + (r - a.H - a.H_kv) * a.v_hs;
        }
        if (!dst && !cache) continue;
        int e0[kEach], e1[kEach];
#pragma unroll
        for (int y = 0; y < kEach; ++y) columns(r, y, &e0[y], &e1[y]);
        if (!is_v) {
            float x[kEach][2 * VEC];
#pragma unroll
            for (int y = 0; y < kEach; ++y) {
                x_lo[y].unpack(x[y]);
                x_hi[y].unpack(x[y] + VEC);
            }
            if (w) {
                uint64_t sq = 0;
#pragma unroll
                for (int y = 0; y < kEach; ++y)
#pragma unroll
                    for (int p = 0; p < 2 * VEC; p += 2) {
                        const uint64_t v = f2_pack(x[y][p], x[y][p + 1]);
                        sq = ffma2(v, v, sq);
                    }
                float ss = f2_lo(sq) + f2_hi(sq);
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(mask, ss, d);
                const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
                const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
                for (int y = 0; y < kEach; ++y) {
                    float ww[2 * VEC];
                    reinterpret_cast<const U *>(w + e0[y])->unpack(ww);
                    reinterpret_cast<const U *>(w + e1[y])->unpack(ww + VEC);
#pragma unroll
                    for (int p = 0; p < 2 * VEC; p += 2) {
                        const uint64_t v = fmul2(fmul2(f2_pack(x[y][p], x[y][p + 1]), inv2), f2_pack(ww[p], ww[p + 1]));
                        x[y][p] = f2_lo(v), x[y][p + 1] = f2_hi(v);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < kEach; ++y) {
                const int first = (u0 + y * kLanes) * VEC;  // pair
                if (first < half) {
                    const float *cs = &cosines[now.k][first], *sn = &sines[now.k][first];
                    auto turn = [&](int p, float &f, float &g) {  // rounded as rope.cu's turn is
                        const float c = cs[p], s = sn[p];
                        const float f2 = fmaf(f, c, -(g * s)), g2 = fmaf(f, s, g * c);
                        // past the last pair nothing is multiplied: 0 times an infinity is none
                        if (first + p < half) f = f2, g = g2;
                    };
                    if (interleaved) {
#pragma unroll
                        for (int p = 0; p < VEC; ++p) turn(p, x[y][2 * p], x[y][2 * p + 1]);
                    } else if (VEC == 1) {
                        turn(0, x[y][0], x[y][VEC]);
                    } else {  // whole units of pairs, two at a time
#pragma unroll
                        for (int p = 0; p < VEC; p += 2) {
                            const uint64_t c = f2_pack(cs[p], cs[p + 1]), s = f2_pack(sn[p], sn[p + 1]);
                            const uint64_t f = f2_pack(x[y][p], x[y][p + 1]), g = f2_pack(x[y][VEC + p], x[y][VEC + p + 1]);
                            const uint64_t f2 = ffma2(f, c, fmul2(fmul2(g, f2_pack(-1.f, -1.f)), s)), g2 = ffma2(f, s, fmul2(g, c));
                            x[y][p] = f2_lo(f2), x[y][p + 1] = f2_hi(f2);
                            x[y][VEC + p] = f2_lo(g2), x[y][VEC + p + 1] = f2_hi(g2);
                        }
                    }
                }
                x_lo[y].pack(x[y]);
                x_hi[y].pack(x[y] + VEC);
            }
        }
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            if (dst) {
                *reinterpret_cast<U *>(dst + e0[y]) = x_lo[y];
                *reinterpret_cast<U *>(dst + e1[y]) = x_hi[y];
            }
            if (cache) {
                *reinterpret_cast<U *>(cache + e0[y]) = x_lo[y];
                *reinterpret_cast<U *>(cache + e1[y]) = x_hi[y];
            }
        }
    }
}

template <typename T, int VEC, int D, bool Interleaved>
cudaError_t launch_t(const NormRopeArgs &a) {
    const int rows = a.H + a.H_kv * (a.append ? 2 : 1);
    const long long sms = a.n_sm > 0 ? a.n_sm : 1;
    // two tokens a block when that still leaves several rounds of blocks an SM;
    // with few tokens the rows of one are split
    int tokens = kTokens;
    while (tokens > 1 && a.T / tokens < 32 * sms) tokens /= 2;
    const long long blocks = (static_cast<long long>(a.T) + tokens - 1) / tokens;
    constexpr int kGroups = kThreads / (D / (2 * VEC) < 32 ? D / (2 * VEC) : 32);
    long long split = (2 * sms + blocks - 1) / blocks;
    const long long most = (rows + kGroups - 1) / kGroups;
    split = split > most ? most : split;
    const int per = static_cast<int>((rows + split - 1) / split);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((rows + per - 1) / per));
    return launch_pdl(norm_rope_kernel<T, VEC, D, Interleaved>, grid, dim3(kThreads), 0, a.stream, a, tokens, per);
}

}  // namespace

template <typename T, int VEC, int D>
static cudaError_t launch_d(const NormRopeArgs &a, bool wide) {
    if (!wide) return launch_t<T, 1, D, false>(a);
    return a.interleaved ? launch_t<T, VEC, D, true>(a) : launch_t<T, VEC, D, false>(a);
}

cudaError_t launch_norm_rope(const NormRopeArgs &a, bool f32, bool wide) {
    if (a.D == 64) return f32 ? launch_d<float, 4, 64>(a, wide) : launch_d<__nv_bfloat16, 8, 64>(a, wide);
    return f32 ? launch_d<float, 4, 128>(a, wide) : launch_d<__nv_bfloat16, 8, 128>(a, wide);
}

}  // namespace attn
