// Attention of a tree of drafted tokens over a KV cache on the sm_103a tensor
// cores (attn_decode_tree, bf16), and the merge of its splits (either type).
//
// Every sequence has T drafted tokens hanging under its committed cache.  Token
// t sees the cache before the draft, itself and its ancestors:
//     out_t = softmax over visible j of (scale q_t . k_j) times v_j.
// The G = H / H_kv query heads of a cached head and the T tokens form the rows
// of 128-row tiles (row r: head r / T, token r % T), so one read of the cache
// serves G T rows; with up to 128 rows the pass over the cache is bound by HBM.
//
// One CTA per (sequence and cached head, split of the keys, row tile), two on
// an SM.  Per tile of 64 keys, as in the grouped decode kernel:
//     S = Q K_j^T  (M 128, N 64, K = D),   O += P V_j  (P from TMEM),
// S double-buffered in TMEM so that the scores of the next tile are computed
// under this tile's softmax.  Splits write their unnormalised O, running max and
// sum in fp32; the merge is exact.  Row tiles of one split are neighbours in the
// grid and read the same keys from L2.
//
// Masks.  Ancestor sets are 128-bit words per token, closed by doubling over the
// parent links while the first tiles are on their way.  Tiles in front of the
// draft carry no mask; the last ones (the edge tiles, at most four) take the
// 64 bits of their keys out of the row's set.  A weight of zero does not hide an
// infinite or NaN value from the second product (0 * inf), and rows past the
// sequence's end hold whatever the cache was left with, so two guard warps pass
// over the V of the edge tiles before their MMA: rows past the end become zeros,
// non-finite elements of drafted rows become zeros which the epilogue adds back
// to the rows that see them.
//
// Roles (8 warps): warp 0 TMA producer (K_j, V_j through a ring), warp 1 TMEM
// allocation and MMA issue, warps 2-5 Q staging, ancestor sets, softmax and
// epilogue (thread = row = TMEM lane), warps 6-7 guard.
#include "kernels.h"
#include "ptx.cuh"
#include "serving.cuh"

namespace attn {
namespace {

constexpr int kN = 64;           // keys per K/V tile
constexpr int kM = 128;          // rows per tile
constexpr int kThreads = 256;
constexpr int kStages = 4;       // K/V ring: 97 KB of shared memory at D = 128, two CTAs an SM
constexpr int kCols = 256;       // TMEM: S buffers at columns 0 and 64, O at 128
constexpr int kEdge = 4;         // tiles of 64 that 128 drafted keys at any offset can touch, and one to spare
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kHugeLog2 = 16777216.0f;  // 2^24

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); }

template <int D>
struct Layout {
    static constexpr int kSub = D / 64;
    static constexpr int kQBlock = kM * 128;
    static constexpr int kKvBlock = kN * 128;
    static constexpr int kKvBytes = kSub * kKvBlock;
    static constexpr int kRingOff = kSub * kQBlock;
    static constexpr int kAncOff = kRingOff + kStages * kKvBytes;
    static constexpr int kBarOff = kAncOff + static_cast<int>(sizeof(Ancestors));
    static constexpr int kSmemBytes = kBarOff + 256 + 1024;
};

struct Bars {
    uint64_t q_full;            // Q staged by the softmax warps
    uint64_t kv_full[kStages];
    uint64_t kv_empty[kStages];
    uint64_t s_full[2];
    uint64_t p_ready[2];
    uint64_t o_done;            // one phase per P V
    uint64_t o_full;
    uint64_t edge_full[kEdge];  // load of the edge tile's V issued
    uint64_t edge_clean[kEdge];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    int spoiled;                // a non-finite value in an edge tile
};
static_assert(sizeof(Bars) <= 256, "barrier block");

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    tree_tc_kernel(const TreeArgs a, const int row_tiles, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv) {
    griddep_launch_dependents();
    griddep_wait();
    using L = Layout<D>;
    const int m = blockIdx.x % row_tiles, c = (blockIdx.x / row_tiles) % a.n_split;
    const int bk = blockIdx.x / row_tiles / a.n_split, b = bk / a.H_kv, g = bk % a.H_kv;
    const int G = a.H / a.H_kv, rows = G * a.T, r0 = m * kM;
    const Draft d = draft_of(a, b);
    const int k0 = c * a.chunk;
    const int nkeys = min(a.chunk, d.L - k0);  // <= 0: nothing here
    if (nkeys <= 0 && a.n_split > 1) return;   // the merge never reads this split
    const int n = nkeys > 0 ? (nkeys + kN - 1) / kN : 0;
    // first tile that some row sees only a part of, or that runs past the end
    const int edge = min(n, max(0, d.past - k0) / kN);

    extern __shared__ __align__(1024) uint8_t dsmem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + L::kRingOff;
    Ancestors &anc = *reinterpret_cast<Ancestors *>(smem + L::kAncOff);
    Bars &bars = *reinterpret_cast<Bars *>(smem + L::kBarOff);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        mbar_init(&bars.q_full, kM);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.kv_full[s], 1);
            mbar_init(&bars.kv_empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.s_full[x], 1);
            mbar_init(&bars.p_ready[x], kM);
        }
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.o_full, 1);
        for (int x = 0; x < kEdge; ++x) {
            mbar_init(&bars.edge_full[x], 1);
            mbar_init(&bars.edge_clean[x], 64);
        }
        mbar_init(&bars.mma_done, 1);
        bars.abort = 0;
        bars.spoiled = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem_base, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;

    if (warp == 0) {
        // ================================================================ TMA producer
        if (lane == 0) {
            prefetch_tmap(&tk);
            prefetch_tmap(&tv);
            bool ok = true;
            int issued = 0;
            for (; issued < 2 * n && ok; ++issued) {
                const int j = issued / 2, kv = issued % 2, s = issued % kStages;
                if (issued >= kStages &&
                    !(ok = mbar_wait(&bars.kv_empty[s], ((issued / kStages) - 1) & 1, &bars.abort)))
                    break;
                mbar_arrive_expect_tx(&bars.kv_full[s], L::kKvBytes);
#pragma unroll
                for (int cb = 0; cb < L::kSub; ++cb)
                    tma_load_3d(ring + s * L::kKvBytes + cb * L::kKvBlock, kv ? &tv : &tk, &bars.kv_full[s], cb * 64,
                                k0 + j * kN, bk);
                if (kv && j >= edge) mbar_arrive(&bars.edge_full[j - edge]);
            }
            // never leave with copies still landing in shared memory
            volatile int never = 0;
            for (int u = max(0, issued - kStages); u < issued; ++u)
                mbar_wait(&bars.kv_full[u % kStages], (u / kStages) & 1, &never);
        }
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        const uint32_t idesc_s = idesc_bf16_f32(kM, kN, 0);
        const uint32_t idesc_o = idesc_bf16_f32(kM, D, 1);
        const uint64_t dq = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t dv0 = sdesc_sw128(smem_u32(ring), L::kKvBlock, 1024);
        auto issue_s = [&](int x, int slot) {
            const uint64_t db = desc_add(dk0, (slot * L::kKvBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss_warp(tmem + static_cast<uint32_t>(x) * kN,
                            desc_add(dq, ((kk / 4) * L::kQBlock + (kk % 4) * 32) >> 4),
                            desc_add(db, ((kk / 4) * L::kKvBlock + (kk % 4) * 32) >> 4), idesc_s, kk > 0);
        };
        auto issue_pv = [&](int x, int slot, bool acc) {
            const uint64_t db = desc_add(dv0, (slot * L::kKvBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
                mma_ts_warp(tmem + 128u, tmem + static_cast<uint32_t>(x) * kN + kk * 8,
                            desc_add(db, (kk * 16 * 128) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u);
        };
        uint32_t pr0 = 0, pr1 = 0;
        bool ok = mbar_wait_warp(&bars.q_full, 0, &bars.abort);
        tc_fence_after();
        // order: S_0 | S_1 PV_0 | S_2 PV_1 | ... | PV_{n-1}; S_j reuses the buffer whose P PV_{j-2} read
        for (int j = 0; j <= n && ok && n > 0; ++j) {
            if (j < n) {
                const int ks = (2 * j) % kStages;
                if (!(ok = mbar_wait_warp(&bars.kv_full[ks], ((2 * j) / kStages) & 1, &bars.abort))) break;
                tc_fence_after();
                issue_s(j & 1, ks);
                tc_commit_warp(&bars.s_full[j & 1]);
                tc_commit_warp(&bars.kv_empty[ks]);
            }
            if (j >= 1) {
                const int t = j - 1, x = t & 1, vs = (2 * t + 1) % kStages;
                if (!(ok = mbar_wait_warp(&bars.kv_full[vs], ((2 * t + 1) / kStages) & 1, &bars.abort))) break;
                if (t >= edge && !(ok = mbar_wait_warp(&bars.edge_clean[t - edge], 0, &bars.abort))) break;
                if (!(ok = mbar_wait_warp(&bars.p_ready[x], x ? pr1 : pr0, &bars.abort))) break;
                if (x) pr1 ^= 1; else pr0 ^= 1;
                tc_fence_after();
                issue_pv(x, vs, t > 0);
                tc_commit_warp(&bars.o_done);
                tc_commit_warp(&bars.kv_empty[vs]);
                if (t == n - 1) tc_commit_warp(&bars.o_full);
            }
        }
        // every MMA must have finished before TMEM is released
        tc_commit_warp(&bars.mma_done);
        volatile int never = 0;
        mbar_wait_warp(&bars.mma_done, 0, &never);
    } else if (warp >= 6) {
        // ================================================================ guard of the edge V tiles
        const int tid = threadIdx.x - 192;
        for (int j = edge; j < n; ++j) {
            const int u = 2 * j + 1, s = u % kStages;
            // the request comes after this use's load was issued, and the stage is
            // not reused before edge_clean: kv_full cannot be a phase off
            if (!mbar_wait_warp<64>(&bars.edge_full[j - edge], 0, &bars.abort)) break;
            if (!mbar_wait_warp(&bars.kv_full[s], (u / kStages) & 1, &bars.abort)) break;
            const uint32_t tile = smem_u32(ring + s * L::kKvBytes);
            const int end = d.L - k0 - j * kN;  // rows of the tile inside the sequence
            bool bad = false;
#pragma unroll 8
            for (int i = tid; i < L::kKvBytes / 16; i += 64) {  // 8 chunks a row, 64 rows a block
                const uint4 v = ld_shared_v4(tile + i * 16);
                if ((i >> 3) % kN >= end) {
                    st_shared_v4(tile + i * 16, 0u, 0u, 0u, 0u);
                } else {
                    const uint32_t n0 = nonfinite2(v.x), n1 = nonfinite2(v.y), n2 = nonfinite2(v.z), n3 = nonfinite2(v.w);
                    if (n0 | n1 | n2 | n3) {
                        bad = true;
                        st_shared_v4(tile + i * 16, v.x & ~n0, v.y & ~n1, v.z & ~n2, v.w & ~n3);
                    }
                }
            }
            if (bad) *static_cast<volatile int *>(&bars.spoiled) = 1;
            fence_proxy_async_shared();
            mbar_arrive(&bars.edge_clean[j - edge]);
        }
    } else {
        // ================================================================ softmax + epilogue
        const int quarter = warp % 4;       // TMEM lanes [32 * quarter, 32 * quarter + 32)
        const int row = quarter * 32 + lane;
        const int tid = threadIdx.x - 64;   // 0 .. 127, for the staging loops
        // Q rows, swizzled as a TMA load would leave them; rows without a token are zeros
#pragma unroll 4
        for (int i = tid; i < kM * D / 8; i += kM) {
            const int rr = i / (D / 8), ch = i % (D / 8), r = r0 + rr;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows && r % a.T < d.n)
                x = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + b * a.q_bs +
                                                     (g * G + r / a.T) * a.q_hs + (r % a.T) * a.q_ts + ch * 8);
            st_shared_v4(smem_u32(smem) + (ch / 8) * L::kQBlock + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), x.x, x.y, x.z,
                         x.w);
        }
        fence_proxy_async_shared();
        mbar_arrive(&bars.q_full);
        build_ancestors(a, b, d, anc, tid, [] { named_bar_sync(1, kM); });
        const int r = r0 + row, t = r % a.T;
        const bool live = r < rows && t < d.n && d.past + t >= 0;
        const uint32_t *set = anc.bits[t];
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const float sl2 = a.scale * kLog2e;
        float m_run = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n && ok; ++j) {
            const int x = j & 1;
            if (!(ok = mbar_wait_warp<32>(&bars.s_full[x], (j >> 1) & 1, &bars.abort))) break;
            tc_fence_after();
            uint32_t s[kN];
            tmem_ld32(t_lane + x * kN, s);
            tmem_ld32(t_lane + x * kN + 32, s + 32);
            tmem_ld_wait();
            reg_fence32(s);
            reg_fence32(s + 32);
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (j >= edge) {
                const int at = k0 + j * kN - d.past;
                see[0] = live ? visible32(set, at) : 0u;
                see[1] = live ? visible32(set, at + 32) : 0u;
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (!(see[e / 32] >> (e % 32) & 1u)) s[e] = f2u(-INFINITY);
            }
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(u2f(s[2 * e]), u2f(s[2 * e + 1]));
#pragma unroll
            for (int cc = 8; cc < kN; cc += 2) m4[(cc / 2) % 4] = fmax3(m4[(cc / 2) % 4], u2f(s[cc]), u2f(s[cc + 1]));
            const float raw = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            const float m_new = fmaxf(m_run, raw == -INFINITY ? -INFINITY : raw * sl2);
            const bool grow = m_new > m_run + kRescaleLog2;
            if (__any_sync(0xffffffffu, grow)) {
                const float factor = grow ? ex2_approx(m_run - m_new) : 1.f;
                if (grow) {
                    l *= factor;
                    m_run = m_new;
                }
                if (j > 0) {
                    // O holds PV_0 .. PV_{j-1}: wait for the last of them
                    if (!(ok = mbar_wait_warp(&bars.o_done, (j - 1) & 1, &bars.abort))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(t_lane + 128 + cc * 32, o);
                        tmem_ld_wait();
                        reg_fence32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = f2u(u2f(o[e]) * factor);
                        tmem_st32(t_lane + 128 + cc * 32, o);
                    }
                }
            }
            const float negm = m_run == -INFINITY ? 0.f : -m_run;  // nothing seen yet: every p below is zero
            float mul = sl2;
            // huge scores: round the product before the difference (as in prefill_tc.cu)
            if (__any_sync(0xffffffffu, negm < -kHugeLog2 || negm > kHugeLog2)) {
#pragma unroll
                for (int e = 0; e < kN; ++e) s[e] = f2u(__fmul_rn(u2f(s[e]), sl2));
                mul = 1.f;
            }
            const uint64_t sl2x2 = f2_pack(mul, mul), negmx2 = f2_pack(negm, negm);
            uint64_t l4[4] = {0, 0, 0, 0};
            uint32_t p[kN / 2];
#pragma unroll
            for (int e = 0; e < kN / 2; ++e) {
                const uint64_t arg = ffma2(f2_pack(u2f(s[2 * e]), u2f(s[2 * e + 1])), sl2x2, negmx2);
                float p0 = ex2_approx(f2_lo(arg)), p1 = ex2_approx(f2_hi(arg));
                if (j >= edge) {  // with a scale of 0 a hidden -inf would become NaN
                    p0 = see[e / 16] >> ((2 * e) % 32) & 1u ? p0 : 0.f;
                    p1 = see[e / 16] >> ((2 * e + 1) % 32) & 1u ? p1 : 0.f;
                }
                l4[e % 4] = fadd2(l4[e % 4], f2_pack(p0, p1));
                // P is rounded to bf16, the operand type of the second product: each
                // weight is off by at most 2^-8 of itself; the sum keeps fp32
                p[e] = pack_bf16x2(p0, p1);
            }
            const uint64_t l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
            l += f2_lo(l2) + f2_hi(l2);
            tmem_st32(t_lane + x * kN, p);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars.p_ready[x]);
        }
        // ---- epilogue
        if (ok && n > 0) {
            ok = mbar_wait_warp(&bars.o_full, 0, &bars.abort);
            tc_fence_after();
        }
        const bool write = ok && r < rows;
        const bool have = live && n > 0;
        const bool spoiled = n > 0 && *static_cast<volatile int *>(&bars.spoiled) != 0 && have;
        const size_t part = (static_cast<size_t>(bk) * rows + r) * a.n_split + c;
        const float inv = 1.f / l;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + b * a.o_bs + (g * G + r / a.T) * a.o_hs + t * a.o_ts;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];  // TMEM of this CTA: loaded unconditionally, used only when valid
            tmem_ld32(t_lane + 128 + cc * 32, o);
            tmem_ld_wait();
            reg_fence32(o);
            if (spoiled) {  // add the non-finite values of the edge tiles that this row sees
                const __nv_bfloat16 *V = static_cast<const __nv_bfloat16 *>(a.v) + static_cast<size_t>(bk) * a.Skv * D + cc * 32;
#pragma unroll 1
                for (int key = k0 + edge * kN; key < k0 + nkeys; ++key) {
                    if (!(visible32(set, key - d.past) & 1u)) continue;
                    const uint32_t *vr = reinterpret_cast<const uint32_t *>(V + static_cast<size_t>(key) * D);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t w = vr[e], nf = nonfinite2(w);
                        if (nf & 0xffffu) o[2 * e] = f2u(u2f(o[2 * e]) + bf16lo_to_f32(w));
                        if (nf & 0xffff0000u) o[2 * e + 1] = f2u(u2f(o[2 * e + 1]) + bf16hi_to_f32(w));
                    }
                }
            }
            if (!write) continue;
            if (a.n_split > 1) {
                float4 *dst = reinterpret_cast<float4 *>(a.part_o + part * D + cc * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(u2f(o[4 * e]), u2f(o[4 * e + 1]), u2f(o[4 * e + 2]), u2f(o[4 * e + 3]));
            } else {
                uint4 *dst = reinterpret_cast<uint4 *>(out + cc * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t pk[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        pk[y] = have ? pack_bf16x2(u2f(o[8 * e + 2 * y]) * inv, u2f(o[8 * e + 2 * y + 1]) * inv) : 0u;
                    dst[e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
        }
        if (write && a.n_split > 1) *reinterpret_cast<float2 *>(a.part_ml + part * 2) = make_float2(m_run, l);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem, kCols);
    }
    if (threadIdx.x == 0 && bars.abort) report_timeout(a.status, 0x44);
}

// ------------------------------------------------------------ merge of the splits

__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// One warp per row: out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c, M the
// largest m_c.  The splits are added in order, so the result does not depend on
// how the CTAs ran.
template <int D, typename T>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int G = a.H / a.H_kv, rows = G * a.T, lane = threadIdx.x % 32;
    const long long R = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
    if (R >= static_cast<long long>(a.B) * a.H_kv * rows) return;
    const int bk = static_cast<int>(R / rows), r = static_cast<int>(R % rows), b = bk / a.H_kv, g = bk % a.H_kv;
    const int t = r % a.T;
    const Draft d = draft_of(a, b);
    const bool live = t < d.n && d.past + t >= 0;
    const int n = live ? (d.L + a.chunk - 1) / a.chunk : 0;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + R * a.n_split;
    const float *po = a.part_o + R * a.n_split * D;
    float M = -INFINITY;
    for (int c = lane; c < n; c += 32) M = fmaxf(M, ml[c].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    const float ref = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    const int col = D == 64 ? 4 * (lane % 16) : 4 * lane;
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
        const float2 x = ml[c];
        const float4 o = *reinterpret_cast<const float4 *>(po + static_cast<size_t>(c) * D + col);
        const float w = ex2_approx(x.x - ref);
        sum = fmaf(w, x.y, sum);
        // a split in which the row saw nothing holds zeros
        acc = make_float4(fmaf(w, o.x, acc.x), fmaf(w, o.y, acc.y), fmaf(w, o.z, acc.z), fmaf(w, o.w, acc.w));
    }
    const float inv = live ? 1.f / sum : 0.f;
    T *out = static_cast<T *>(a.out) + b * a.o_bs + (g * G + r / a.T) * a.o_hs + t * a.o_ts;
    if (lane < D / 4) store4(out + col, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

template <int D>
cudaError_t launch_tree_t(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv) {
    using L = Layout<D>;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int row_tiles = ((a.H / a.H_kv) * a.T + kM - 1) / kM;
    const unsigned grid = static_cast<unsigned>(a.B * a.H_kv) * a.n_split * row_tiles;
    e = launch_pdl(tree_tc_kernel<D>, dim3(grid), dim3(kThreads), L::kSmemBytes, a.stream, a, row_tiles, tk, tv);
    if (e != cudaSuccess || a.n_split == 1) return e;
    return launch_tree_combine(a, false);
}

}  // namespace

int tree_chunk(int B, int H, int H_kv, int T, int Skv, bool f32, int n_sm) {
    // several waves of the CTAs an SM holds, at least a few tiles each
    const int rows = (H / H_kv) * T, per_tile = f32 ? 32 : kM;
    const long long units = static_cast<long long>(B) * H_kv * ((rows + per_tile - 1) / per_tile);
    const long long tiles = (static_cast<long long>(Skv) + kN - 1) / kN;
    const long long want = 6LL * 2 * (n_sm > 0 ? n_sm : 1);
    long long per = (units * tiles + want - 1) / want;
    const long long least = f32 ? 2 : 8;
    per = per < least ? least : per;
    per = per > tiles ? tiles : per;
    per = per < 1 ? 1 : per;
    return static_cast<int>(per * kN);
}

cudaError_t launch_tree_tc(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv) {
    return a.D == 64 ? launch_tree_t<64>(a, tk, tv) : launch_tree_t<128>(a, tk, tv);
}

cudaError_t launch_tree_combine(const TreeArgs &a, bool f32) {
    const long long R = static_cast<long long>(a.B) * a.H * a.T;
    const dim3 grid(static_cast<unsigned>((R + 7) / 8));
    if (a.D == 64)
        return f32 ? launch_pdl(tree_merge_kernel<64, float>, grid, dim3(256), 0, a.stream, a)
                   : launch_pdl(tree_merge_kernel<64, __nv_bfloat16>, grid, dim3(256), 0, a.stream, a);
    return f32 ? launch_pdl(tree_merge_kernel<128, float>, grid, dim3(256), 0, a.stream, a)
               : launch_pdl(tree_merge_kernel<128, __nv_bfloat16>, grid, dim3(256), 0, a.stream, a);
}

}  // namespace attn
