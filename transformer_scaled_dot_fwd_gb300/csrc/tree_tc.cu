// Attention of a tree of drafted tokens over a KV cache on the sm_103a tensor
// cores (attn_decode_tree, bf16), and the merges of its partial results.
//
// Every sequence has T drafted tokens hanging under its committed cache.  Token
// t sees the cache before the draft, itself and its ancestors:
//     out_t = softmax over visible j of (scale q_t . k_j) times v_j.
// The G = H / H_kv query heads of a cached head and the T tokens form the rows
// of 128-row tiles (row r: head r / T, token r % T), so one read of the cache
// serves G T rows; with up to 128 rows the pass over the cache is bound by HBM.
//
// Work split.  A unit is a cached head of a sequence with one or two of its row
// tiles, its cost the number of its 128-key tiles.  One persistent CTA per SM
// takes an equal run of the list of all units' tiles, whatever the lengths are:
// no tail, and at most two units per CTA are shared with neighbours.  Those
// leave their unnormalised O, running max and sum in fp32 in the CTA's slots of
// the workspace, for a merge in the order of the keys; whole units are written
// out directly.
//
// Two softmax warpgroups (streams) keep two S and two O accumulators in TMEM
// busy.  A unit with two row tiles gives each stream one of them, and both read
// the same K/V tiles.  A unit with one row tile gives the streams alternate K/V
// tiles; they join their O, max and sum at the end of the unit's run.  Order:
//     two tiles:  S0_0 S1_0 | PV0_j S0_{j+1} PV1_j S1_{j+1} | ...
//     one tile:   S0_0 S1_1 | PV_j S_{j+2} (stream j & 1)   | ...
// so that a stream always has the other's MMAs to hide behind.
//
// Masks.  Ancestor sets are 128-bit words per token, closed by doubling over the
// parent links.  Tiles in front of the draft carry no mask; the last ones (the
// edge tiles, at most three) take the 128 bits of their keys out of the row's set.  A
// weight of zero does not hide an infinite or NaN value from the second product
// (0 * inf), and rows past the sequence's end hold whatever the cache was left
// with, so two guard warps pass over the V of the edge tiles before their MMA:
// rows past the end become zeros, non-finite elements of drafted rows become
// zeros which the epilogue adds back to the rows that see them.
//
// Measured (H 32, H_kv 8, D 128): 16 sequences of 2000-8192 rows, up to 24 drafts
// (323 MB to read): 63 us, of it 49 us at 6.6 TB/s between the first and the last
// tile, 4 us the merge.  64 sequences of 4096-8192 rows, 63 drafts (1.69 GB, 407
// GFLOP): 314-348 us, 1170-1295 TFLOP/s by the power limit, a pair of tiles in 1.7 us.  One sequence
// of 1500 rows, 8 drafts: 12 us (12.8 a call).  The first form, splits of a fixed number of keys
// with a CTA and one stream each, two to an SM, took 98, 526 and 14 us: a single
// stream waits for its own MMAs.
//
// Roles (12 warps): warp 0 walks the CTA's run and loads K_j, V_j through a ring
// of 128-row TMA tiles, warp 1 allocates TMEM and issues the MMAs, warps 2-3
// stage the next unit's Q and ancestor sets while the streams finish the last
// one (the streams stage the first), and guard, warps 4-7 and 8-11 are the streams (softmax, epilogue; thread =
// row = TMEM lane).
#include "kernels.h"
#include "ptx.cuh"
#include "serving.cuh"

namespace attn {
namespace {

constexpr int kN = 128;          // keys per K/V tile
constexpr int kM = 128;          // rows per tile
constexpr int kThreads = 384;
constexpr uint32_t kRegsOther = 64;     // warps 0-3 after setmaxnreg
constexpr uint32_t kRegsSoftmax = 216;  // warps 4-11: 128 * 64 + 256 * 216 <= 384 * 168
constexpr int kTmemCols = 512;   // S0 0, S1 128, O0 256, O1 256 + D
constexpr int kRing = 4;         // unit runs in flight between the roles
constexpr int kRingReaders = 32 + 256;
// Requests to warps 2-3: one per run and one per edge tile.  No more than kRing
// runs are open at once, and an edge tile holds a K/V stage: fewer than 16 in all.
constexpr int kGuardRing = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kHugeLog2 = 16777216.0f;  // 2^24
// Fewest tiles a CTA takes: below it a run costs more to start and merge than to
// compute (1, 2, 3, 4 and 6 tiles: 16.7, 14.1, 14.0, 14.4 and 15.5 us for one
// sequence of 1500 rows).
#ifndef ATTN_TREE_MIN_TILES
#define ATTN_TREE_MIN_TILES 2
#endif
// What a unit costs beside its tiles, in tiles: start, epilogue, merge (0, 2, 4, 6
// and 8: 65.7, 64.7, 62.9, 62.9 and 63.5 us for the 16 sequences).
#ifndef ATTN_TREE_UNIT_COST
#define ATTN_TREE_UNIT_COST 5
#endif

constexpr int kUnitCost = ATTN_TREE_UNIT_COST, kMinCost = ATTN_TREE_MIN_TILES;

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

// A run of K/V tiles [j0, j0 + n) of one unit.
struct Run {
    int b, bk;      // sequence, sequence and cached head
    int tile;       // first row tile
    int j0, n;      // n < 0: no more work
    int slot;       // workspace slot, -1: the whole unit, written out
    int L, nd, past;
};

struct GuardReq {
    int stage;   // K/V stage of an edge tile, kStageRun: a new run, kEnd: no more work
    int parity;  // of the stage's kv_full
    int rows;    // rows of the tile inside the sequence
    int run;     // ring slot
};
constexpr int kEnd = -1, kStageRun = -2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Single: one row tile in all, its second Q buffer is one more K/V stage.
template <int D, bool Single>
struct Layout {
    static constexpr int kSub = D / 64;
    static constexpr int kBlock = 128 * 128;        // 128 rows x 128 bytes
    static constexpr int kTile = kSub * kBlock;
    static constexpr int kQTiles = Single ? 1 : 2;
    static constexpr int kStages = D == 128 ? (Single ? 5 : 4) : 8;
    static constexpr int kRingOff = kQTiles * kTile;
    static constexpr int kAncOff = kRingOff + kStages * kTile;
    static constexpr int kExOff = kAncOff + 2 * static_cast<int>(sizeof(Ancestors));
    static constexpr int kBarOff = kExOff + 256 * 8;
    static constexpr int kSmemBytes = kBarOff + 1024 + 1024;
};

struct Bars {
    uint64_t q_full[2];         // Q and ancestor sets of run k staged: [k & 1]
    uint64_t q_first;           // Q of run 0 staged, by the streams
    uint64_t q_free;            // a run's last S MMA is complete
    uint64_t kv_full[8], kv_empty[8];
    uint64_t s_full[2], p_ready[2], o_full[2];
    uint64_t run_full[kRing], run_empty[kRing];
    uint64_t guard_full[kGuardRing], guard_clean[kGuardRing];
    uint64_t join;              // both streams (a barrier with a limit)
    uint64_t mma_done;
    Run run[kRing];
    GuardReq req[kGuardRing];
    int spoiled[kRing];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// Every unit has at least one tile, so that the rows of empty sequences are
// written (as zeros) like the others.
__device__ __forceinline__ int tiles_of(const Draft &d) { return max(1, (d.L + kN - 1) / kN); }
__device__ __forceinline__ int cost_of(const Draft &d) { return tiles_of(d) + kUnitCost; }

__device__ __forceinline__ Run read_run(Bars &bars, int slot) {
    const volatile Run &s = bars.run[slot];
    return Run{s.b, s.bk, s.tile, s.j0, s.n, s.slot, s.L, s.nd, s.past};
}
__device__ __forceinline__ bool take_run(Bars &bars, int k, Run *r) {
    if (!mbar_wait_warp(&bars.run_full[k % kRing], (k / kRing) & 1, &bars.abort)) return false;
    *r = read_run(bars, k % kRing);
    return true;
}

// First edge tile of a run, relative to j0: a tile that some row sees only a
// part of, or that runs past the end.
__device__ __forceinline__ int edge_of(const Run &r) { return min(r.n, max(0, max(0, r.past) / kN - r.j0)); }

// Q rows of a run's row tiles into shared memory at `dst`, as a TMA load would
// leave them (128-byte swizzle); rows without a token are zeros.  D / 8 threads
// share a row; a thread's rows are kStep apart, so its place in the swizzle
// pattern of 8 rows takes 8 / kStep values in turn (one, if kStep >= 8).
template <int D, int Threads>
__device__ __forceinline__ void stage_q(const TreeArgs &a, const Run &r, int tiles, uint32_t dst, int tid) {
    constexpr int kBlock = 128 * 128, kTile = D / 64 * kBlock;
    constexpr int kChunks = D / 8, kStep = Threads / kChunks;  // 16-byte chunks of a row; rows a pass
    constexpr int kPass = kStep < 8 ? 8 : kStep;               // rows of the inner loop
    const int G = a.H / a.H_kv, ch = tid % kChunks, r0 = tid / kChunks, q0 = r.tile * kM + r0;
    int t = q0 % a.T, left = G * a.T - q0;
    const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(a.q) + r.b * a.q_bs +
                             static_cast<long long>((r.bk - r.b * a.H_kv) * G + q0 / a.T) * a.q_hs + t * a.q_ts + ch * 8;
    const long long step = kStep * a.q_ts, wrap = a.q_hs - a.T * a.q_ts;
    dst += (ch / 8) * kBlock + r0 * 128;
    for (int rr = 0; rr < tiles * kM; rr += kPass) {
        if (rr == kM) dst += kTile - kBlock;
#pragma unroll
        for (int e = 0; e < kPass; e += kStep) {
            const bool in = left > 0 && t < r.nd;
            cp_async16(dst + (((ch & 7) ^ ((r0 + e) & 7)) << 4), in ? Q : static_cast<const __nv_bfloat16 *>(a.q),
                       in ? 16u : 0u);
            dst += kStep * 128;
            left -= kStep;
            t += kStep;
            Q += step;
            while (t >= a.T) t -= a.T, Q += wrap;
        }
    }
    cp_async_wait_all();
    fence_proxy_async_shared();
}

template <int D, bool Single>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const TreeArgs a, const int row_tiles, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv) {
    using L = Layout<D, Single>;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + L::kRingOff;
    Ancestors *anc = reinterpret_cast<Ancestors *>(smem + L::kAncOff);  // [run & 1]
    float2 *ex = reinterpret_cast<float2 *>(smem + L::kExOff);  // [stream][row] max, sum
    Bars &bars = *reinterpret_cast<Bars *>(smem + L::kBarOff);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int G = a.H / a.H_kv, rows = G * a.T;
    const int pairs = (row_tiles + 1) / 2;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        for (int x = 0; x < 2; ++x) mbar_init(&bars.q_full[x], 64);
        mbar_init(&bars.q_first, 256);
        mbar_init(&bars.q_free, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.kv_full[s], 1);
            mbar_init(&bars.kv_empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.s_full[x], 1);
            mbar_init(&bars.p_ready[x], kM);
            mbar_init(&bars.o_full[x], 1);
        }
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&bars.run_full[s], 1);
            mbar_init(&bars.run_empty[s], kRingReaders);
        }
        for (int s = 0; s < kGuardRing; ++s) {
            mbar_init(&bars.guard_full[s], 1);
            mbar_init(&bars.guard_clean[s], 2);  // guard warps
        }
        mbar_init(&bars.join, 256);
        mbar_init(&bars.mma_done, 1);
        bars.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    griddep_launch_dependents();
    griddep_wait();

    if (warp == 0) {
        // ================================================================ walk and TMA loads
        regs_dec<kRegsOther>();
        const int per = a.H_kv * pairs;  // units of a sequence
        int total = 0;                   // cost of all units (the host has checked that it fits)
        Draft mine{0, 0, 0};             // of sequence b0 + lane
        for (int b0 = lane; b0 < a.B; b0 += 32) {
            mine = draft_of(a, b0);
            total += cost_of(mine);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        total *= per;
        // CTA i of N takes [total i / N, total (i + 1) / N) of the units' costs laid end to
        // end; a unit's tiles come first in its share, so a cut in the rest falls between units
        const int most = (total + kMinCost - 1) / kMinCost;
        const int N = min(most, static_cast<int>(gridDim.x)), I = blockIdx.x;
        const bool idle = I >= N;
        const int each = total / N, odd = total % N;
        const int lo = idle ? 0 : each * I + odd * I / N, hi = idle ? 0 : each * (I + 1) + odd * (I + 1) / N;
        // sequence that holds position lo, and the first position of its units
        int b = 0, base = 0;
        for (int b0 = 0; !idle && b0 < a.B; b0 += 32) {
            if (a.B > 32) mine = draft_of(a, min(b0 + lane, a.B - 1));
            const int t = b0 + lane < a.B ? cost_of(mine) * per : 0;
            int sum = t;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, base + sum > lo);
            if (past) {
                const int f = __ffs(past) - 1;
                b = b0 + f;
                base += __shfl_sync(0xffffffffu, sum - t, f);
                break;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        Draft d{__shfl_sync(0xffffffffu, mine.L, b % 32), __shfl_sync(0xffffffffu, mine.n, b % 32), 0};
        d.past = d.L - d.n;
        if (lane == 0) {
            int issued = 0, requests = 0, k = 0;
            bool ok = true;
            int4 rec = make_int4(-1, 0, 0, 0), rec2 = make_int4(0, 0, 0, 0);
            int nt = tiles_of(d);
            int u = (lo - base) / cost_of(d), j = (lo - base) % cost_of(d);
            int pos = lo;  // of tile j of unit u
            auto next_unit = [&] {
                pos += cost_of(d) - j;
                j = 0;
                if (++u == per) {
                    u = 0;
                    if (++b < a.B) {
                        d = draft_of(a, b);
                        nt = tiles_of(d);
                    }
                }
            };
            if (j >= nt) next_unit();
            while (ok) {
                const int slot = k % kRing;
                if (k >= kRing && !(ok = mbar_wait(&bars.run_empty[slot], ((k / kRing) - 1) & 1, &bars.abort))) break;
                Run r{0, 0, 0, 0, -1, 0, 0, 0, 0};
                if (pos < hi) {
                    r.b = b;
                    r.bk = b * a.H_kv + u / pairs;
                    r.tile = 2 * (u % pairs);
                    r.j0 = j;
                    r.n = min(nt - j, hi - pos);
                    r.slot = r.n == nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (j == 0 ? 1 : 0);
                    r.L = d.L, r.nd = d.n, r.past = d.past;
                    if (j == 0 && r.n < nt) {  // the unit begins here and goes on in CTAs up to rec.w
                        const long long last = pos + nt - 1;
                        rec = make_int4(r.bk, r.tile, b, static_cast<int>(((last + 1) * N - 1) / total));  // its CTA
                        rec2 = make_int4(d.n, d.past, 0, 0);
                    }
                }
                volatile Run &w = bars.run[slot];
                w.b = r.b, w.bk = r.bk, w.tile = r.tile, w.j0 = r.j0, w.n = r.n, w.slot = r.slot;
                w.L = r.L, w.nd = r.nd, w.past = r.past;
                *static_cast<volatile int *>(&bars.spoiled[slot]) = 0;
                mbar_arrive(&bars.run_full[slot]);
                if (r.n < 0) break;
                auto request = [&](int stage, int parity, int inside) {
                    volatile GuardReq &q = bars.req[requests % kGuardRing];
                    q.stage = stage, q.parity = parity, q.rows = inside, q.run = slot;
                    mbar_arrive(&bars.guard_full[requests % kGuardRing]);
                    ++requests;
                };
                request(kStageRun, 0, 0);
                const int edge = edge_of(r);
                auto load = [&](int jj, int kv) {
                    if (!ok || jj >= r.n) return;
                    const int s = issued % kStages;
                    if (issued >= kStages && !(ok = mbar_wait(&bars.kv_empty[s], ((issued / kStages) - 1) & 1, &bars.abort)))
                        return;
                    mbar_arrive_expect_tx(&bars.kv_full[s], L::kTile);
#pragma unroll
                    for (int c = 0; c < L::kSub; ++c)
                        tma_load_3d(ring + s * L::kTile + c * L::kBlock, kv ? &tv : &tk, &bars.kv_full[s], c * 64,
                                    (r.j0 + jj) * kN, r.bk);
                    if (kv && jj >= edge) request(s, (issued / kStages) & 1, r.L - (r.j0 + jj) * kN);
                    ++issued;
                };
                // at the start Q goes before all but the first K on the way from memory
                auto q_before = [&] {
                    if (k == 0 && ok) ok = mbar_wait(&bars.q_first, 0, &bars.abort);
                };
                if (Single || r.tile + 1 >= row_tiles) {  // one row tile: K0 K1 | V0 K2 | V1 K3 | ...
                    load(0, 0);
                    q_before();
                    load(1, 0);
                    for (int jj = 0; jj < r.n && ok; ++jj) {
                        load(jj, 1);
                        load(jj + 2, 0);
                    }
                } else {
                    for (int jj = 0; jj < r.n && ok; ++jj) {
                        load(jj, 0);
                        if (jj == 0) q_before();
                        load(jj, 1);
                    }
                }
                ++k;
                if (r.j0 + r.n == nt)
                    next_unit();
                else
                    pos = hi;
            }
            if (ok) {  // no more work for the guard
                *static_cast<volatile int *>(&bars.req[requests % kGuardRing].stage) = kEnd;
                mbar_arrive(&bars.guard_full[requests % kGuardRing]);
            }
            int4 *out = reinterpret_cast<int4 *>(a.merge) + 2 * blockIdx.x;
            out[0] = rec;
            out[1] = rec2;
            // never leave with copies still landing in shared memory
            volatile int never = 0;
            for (int x = max(0, issued - kStages); x < issued; ++x)
                mbar_wait(&bars.kv_full[x % kStages], (x / kStages) & 1, &never);
        }
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        regs_dec<kRegsOther>();
        const uint32_t idesc_s = idesc_bf16_f32(kM, kN, 0);
        const uint32_t idesc_o = idesc_bf16_f32(kM, D, 1);
        const uint64_t dq0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t dv0 = sdesc_sw128(smem_u32(ring), L::kBlock, 1024);
        auto issue_s = [&](int x, int qbuf, int slot) {  // S_x = Q_qbuf K^T
            const uint64_t da = desc_add(dq0, (qbuf * L::kTile) >> 4), db = desc_add(dk0, (slot * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk / 4) * L::kBlock + (kk % 4) * 32) >> 4;
                mma_ss_warp(tmem + x * 128u, desc_add(da, off), desc_add(db, off), idesc_s, kk > 0);
            }
        };
        auto issue_pv = [&](int x, int slot, bool acc) {  // O_x (+)= P_x V
            const uint64_t db = desc_add(dv0, (slot * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
                mma_ts_warp(tmem + 256u + x * static_cast<uint32_t>(D), tmem + x * 128u + kk * 8,
                            desc_add(db, (kk * 16 * 128) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u);
        };
        int consumed = 0, cleaned = 0;
        uint32_t pr[2] = {0, 0};
        bool ok = true;
        auto next_stage = [&](int *slot) {  // wait for the next ring stage
            *slot = consumed % kStages;
            if (!(ok = mbar_wait_warp(&bars.kv_full[*slot], (consumed / kStages) & 1, &bars.abort))) return;
            ++consumed;
        };
        auto guarded = [&](bool edge) {
            if (!edge) return;
            if ((ok = mbar_wait_warp(&bars.guard_clean[cleaned % kGuardRing], (cleaned / kGuardRing) & 1, &bars.abort)))
                ++cleaned;
        };
        for (int k = 0; ok; ++k) {
            Run r;
            if (!(ok = take_run(bars, k, &r))) break;
            mbar_arrive(&bars.run_empty[k % kRing]);
            const int n = __shfl_sync(0xffffffffu, r.n, 0);
            if (n < 0) break;
            const int edge = __shfl_sync(0xffffffffu, edge_of(r), 0);
            const bool one = Single || __shfl_sync(0xffffffffu, r.tile, 0) + 1 >= row_tiles;
            if (!(ok = mbar_wait_warp(k == 0 ? &bars.q_first : &bars.q_full[k & 1], (k >> 1) & 1, &bars.abort))) break;
            int ks = 0, vs = 0;
            if (one) {
                // stream x = tile & 1, both on Q buffer 0
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (x >= n) break;
                    next_stage(&ks);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(x, 0, ks);
                    tc_commit_warp(&bars.s_full[x]);
                    tc_commit_warp(&bars.kv_empty[ks]);
                    if (x + 1 == n) tc_commit_warp(&bars.q_free);
                }
                auto step = [&](int j, int x) {
                    next_stage(&vs);
                    if (ok) guarded(j >= edge);
                    if (!ok || !(ok = mbar_wait_warp(&bars.p_ready[x], pr[x], &bars.abort))) return;
                    pr[x] ^= 1;
                    tc_fence_after();
                    issue_pv(x, vs, j >= 2);
                    if (j + 2 >= n) tc_commit_warp(&bars.o_full[x]);
                    tc_commit_warp(&bars.kv_empty[vs]);
                    if (j + 2 < n) {
                        next_stage(&ks);
                        if (!ok) return;
                        tc_fence_after();
                        issue_s(x, 0, ks);
                        tc_commit_warp(&bars.s_full[x]);
                        tc_commit_warp(&bars.kv_empty[ks]);
                        if (j + 3 == n) tc_commit_warp(&bars.q_free);  // the last S of the run
                    }
                };
                for (int j = 0; j < n && ok; j += 2) {
                    step(j, 0);
                    if (ok && j + 1 < n) step(j + 1, 1);
                }
            } else {
                next_stage(&ks);
                if (!ok) break;
                tc_fence_after();
                issue_s(0, 0, ks);
                tc_commit_warp(&bars.s_full[0]);
                issue_s(1, L::kQTiles - 1, ks);
                tc_commit_warp(&bars.s_full[1]);
                tc_commit_warp(&bars.kv_empty[ks]);
                if (n == 1) tc_commit_warp(&bars.q_free);
                for (int j = 0; j < n && ok; ++j) {
                    next_stage(&vs);
                    if (ok) guarded(j >= edge);
                    if (!ok || !(ok = mbar_wait_warp(&bars.p_ready[0], pr[0], &bars.abort))) break;
                    pr[0] ^= 1;
                    tc_fence_after();
                    issue_pv(0, vs, j > 0);
                    const bool next = j + 1 < n;
                    if (!next) tc_commit_warp(&bars.o_full[0]);
                    if (next) {
                        next_stage(&ks);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(0, 0, ks);
                        tc_commit_warp(&bars.s_full[0]);
                    }
                    if (!(ok = mbar_wait_warp(&bars.p_ready[1], pr[1], &bars.abort))) break;
                    pr[1] ^= 1;
                    tc_fence_after();
                    issue_pv(1, vs, j > 0);
                    if (!next) tc_commit_warp(&bars.o_full[1]);
                    tc_commit_warp(&bars.kv_empty[vs]);
                    if (next) {
                        issue_s(1, L::kQTiles - 1, ks);
                        tc_commit_warp(&bars.s_full[1]);
                        tc_commit_warp(&bars.kv_empty[ks]);
                        if (j + 2 == n) tc_commit_warp(&bars.q_free);
                    }
                }
            }
        }
        // every MMA must have finished before TMEM is released
        tc_commit_warp(&bars.mma_done);
        volatile int never = 0;
        mbar_wait_warp(&bars.mma_done, 0, &never);
    } else if (warp < 4) {
        // ================================================================ Q, ancestor sets, guard of the edge V tiles
        regs_dec<kRegsOther>();
        const int tid = threadIdx.x - 64;
        bool ok = true;
        // Run k, in ring slot `slot`.  Its set buffer was last read by run k - 2, its Q
        // buffers by the S MMAs of run k - 1.
        auto stage_run = [&](int k, int slot) {
            const Run r = read_run(bars, slot);
            if (k >= 2 && !(ok = mbar_wait_warp<64>(&bars.run_empty[(k - 2) % kRing], ((k - 2) / kRing) & 1, &bars.abort)))
                return;
            // warp 2 alone closes the sets: a warp's barrier is cheaper than one of two warps
            if (warp == 2 && edge_of(r) < r.n)
                build_ancestors<32>(a, r.b, Draft{r.L, r.nd, r.past}, anc[k & 1], lane, [] { __syncwarp(); });
            if (k >= 1) {
                if (!(ok = mbar_wait_warp<64>(&bars.q_free, (k - 1) & 1, &bars.abort))) return;
                stage_q<D, 64>(a, r, Single || r.tile + 1 >= row_tiles ? 1 : 2, smem_u32(smem), tid);
            }
            mbar_arrive(&bars.q_full[k & 1]);
        };
        for (int q = 0, k = 0, edges = 0; ok; ++q) {
            const int slot = q % kGuardRing;
            // a request comes after its load was issued, and its stage is not reused
            // before guard_clean: kv_full cannot be a phase off
            if (!mbar_wait_warp<64>(&bars.guard_full[slot], (q / kGuardRing) & 1, &bars.abort)) break;
            const volatile GuardReq &rq = bars.req[slot];
            const int stage = rq.stage, parity = rq.parity, inside = rq.rows, run = rq.run;
            if (stage == kStageRun) {
                stage_run(k++, run);
                continue;
            }
            if (stage < 0) break;
            if (!mbar_wait_warp(&bars.kv_full[stage], parity, &bars.abort)) break;
            const uint32_t tile = smem_u32(ring + stage * L::kTile);
            const bool bad = clean_v_tile<L::kSub, kN, 64>(tile, inside, tid);
            if (bad) *static_cast<volatile int *>(&bars.spoiled[run]) = 1;
            if (inside < kN || __any_sync(0xffffffffu, bad)) fence_proxy_async_shared();  // written: the MMA must see it
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.guard_clean[edges % kGuardRing]);  // edge tiles are counted by themselves
            ++edges;
        }
    } else {
        // ================================================================ softmax streams
        regs_inc<kRegsSoftmax>();
        const int x = (warp - 4) / 4;
        const int quarter = warp % 4;  // TMEM lanes [32 * quarter, 32 * quarter + 32)
        const int row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_s = t_lane + x * 128u, t_o = t_lane + 256u + x * static_cast<uint32_t>(D);
        const float sl2 = a.scale * kLog2e;
        uint32_t sp = 0, o_uses[2] = {0, 0};
        bool ok = true;
        uint32_t joins = 0;
        auto join = [&] {  // waits for all threads of both streams, or for the abort flag
            mbar_arrive(&bars.join);
            ok = mbar_wait_warp(&bars.join, joins & 1, &bars.abort) && ok;
            ++joins;
        };
        for (int k = 0; ok; ++k) {
            bool one, live;
            int n, edge, at0;  // tiles of this stream, first edge tile, draft-relative first key of the run
            const uint32_t *set;
            {
                Run r;
                if (!(ok = take_run(bars, k, &r))) break;
                if (r.n < 0) break;
                one = Single || r.tile + 1 >= row_tiles;
                edge = edge_of(r);
                const int q = (r.tile + (one ? 0 : x)) * kM + row;  // this thread's row of the unit
                const int t = q % a.T;
                live = q < rows && t < r.nd && r.past + t >= 0;
                set = anc[k & 1].bits[t];
                n = one ? (r.n - x + 1) / 2 : r.n;
                at0 = r.j0 * kN - r.past;
                if (k == 0) {  // nothing else to do yet
                    stage_q<D, 256>(a, r, one ? 1 : 2, smem_u32(smem), threadIdx.x - 128);
                    mbar_arrive(&bars.q_first);
                }
            }
            // the ancestor sets (and Q) of this run
            if (!(ok = mbar_wait_warp<32>(&bars.q_full[k & 1], (k >> 1) & 1, &bars.abort))) break;
            float m_run = -INFINITY, l = 0.f;
            bool huge = sl2 == 0.f;  // some row of the warp is
            for (int i = 0; i < n; ++i) {
                const int j = one ? 2 * i + x : i;
                if (!(ok = mbar_wait_warp<32>(&bars.s_full[x], sp, &bars.abort))) break;
                sp ^= 1;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, s + c * 32);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_fence32(s + c * 32);
                const bool masked = j >= edge;
                if (masked) {
                    const int at = at0 + j * kN;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t see = live ? visible32(set, at + 32 * c) : 0u;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see >> e & 1u)) s[32 * c + e] = f2u(-INFINITY);
                    }
                }
                float m8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) m8[e] = fmaxf(u2f(s[2 * e]), u2f(s[2 * e + 1]));
#pragma unroll
                for (int c = 16; c < 128; c += 2) m8[(c / 2) % 8] = fmax3(m8[(c / 2) % 8], u2f(s[c]), u2f(s[c + 1]));
                const float raw = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
                const float m_new = fmaxf(m_run, raw == -INFINITY ? -INFINITY : raw * sl2);
                const bool grow = m_new > m_run + kRescaleLog2;
                float mul = sl2;
                if (__any_sync(0xffffffffu, grow || huge)) {
                    const float factor = grow ? ex2_approx(m_run - m_new) : 1.f;
                    if (grow) {
                        l *= factor;
                        m_run = m_new;
                    }
                    // huge scores: round the product before the difference (as in prefill_tc.cu); a
                    // scale of 0: a hidden key's -inf must not become NaN.  A row without them
                    // has its product there and here a factor of 1: another row's scores do not
                    // change its bits.
                    const bool mine = sl2 == 0.f || (fabsf(m_run) > kHugeLog2 && m_run != -INFINITY);
                    huge = __any_sync(0xffffffffu, mine);
                    if (huge) {
                        const int at = at0 + j * kN;
                        const float first = mine ? sl2 : 1.f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t see = !masked ? 0xffffffffu : live ? visible32(set, at + 32 * c) : 0u;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[32 * c + e] = see >> e & 1u ? f2u(__fmul_rn(u2f(s[32 * c + e]), first)) : f2u(-INFINITY);
                        }
                        mul = mine ? 1.f : sl2;
                    }
                    if (i > 0 && __any_sync(0xffffffffu, grow)) {  // this stream's earlier P V are complete: S was issued after them
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(t_o + c * 32, o);
                            tmem_ld_wait();
                            reg_fence32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = f2u(u2f(o[e]) * factor);
                            tmem_st32(t_o + c * 32, o);
                        }
                    }
                }
                const float negm = m_run == -INFINITY ? 0.f : -m_run;  // nothing seen yet: every p below is zero
                const uint64_t mul2 = f2_pack(mul, mul), negm2 = f2_pack(negm, negm);
                uint64_t l4[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 64 * h + 2 * e;
                        const uint64_t arg = ffma2(f2_pack(u2f(s[c]), u2f(s[c + 1])), mul2, negm2);
                        const float p0 = ex2_approx(f2_lo(arg)), p1 = ex2_approx(f2_hi(arg));
                        l4[e % 4] = fadd2(l4[e % 4], f2_pack(p0, p1));
                        // P is rounded to bf16, the operand type of the second product: each
                        // weight is off by at most 2^-8 of itself; the sum keeps fp32
                        p[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32(t_s + h * 32, p);
                }
                const uint64_t l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
                l += f2_lo(l2) + f2_hi(l2);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars.p_ready[x]);
            }
            // ---- epilogue (the run again, from its ring slot: nothing of it stays live above)
            const Run r = read_run(bars, k % kRing);
            const int q = (r.tile + (one ? 0 : x)) * kM + row, t = q % a.T;
            const bool other = one && r.n > 1;  // the other stream has a part of the same rows
            float w = 1.f, w_other = 0.f, m = m_run, sum = l;
            if (one) {
                ex[x * kM + row] = make_float2(m_run, l);
                join();
                const float2 y = ex[(x ^ 1) * kM + row];
                m = fmaxf(m_run, y.x);
                const float ref = m == -INFINITY ? 0.f : m;
                w = ex2_approx(m_run - ref);
                w_other = ex2_approx(y.x - ref);
                sum = l * w + y.y * w_other;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const bool used = one ? y < r.n : true;
                if (used && (one || y == x) && ok) ok = mbar_wait_warp(&bars.o_full[y], o_uses[y] & 1, &bars.abort);
                if (used) ++o_uses[y];
            }
            tc_fence_after();
            const bool write = ok && q < rows;
            const bool spoiled = *static_cast<volatile int *>(&bars.spoiled[k % kRing]) != 0 && live;
            const float inv = 1.f / sum;
            constexpr int slot_rows = L::kQTiles * kM;
            const int slot_row = (one ? 0 : x * kM) + row;
            // a unit of one row tile: stream 0 writes the first half of the columns, stream 1 the second
            const int c0 = one ? x * (D / 64) : 0, c1 = one ? c0 + D / 64 : D / 32;
            const int h = (r.bk - r.b * a.H_kv) * G + q / a.T;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + r.b * a.o_bs + h * a.o_hs + t * a.o_ts;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                __syncwarp();
                uint32_t o[32];  // TMEM of this CTA: loaded unconditionally, used only when valid
                tmem_ld32((one ? t_lane + 256u : t_o) + c * 32, o);
                tmem_ld_wait();
                reg_fence32(o);
                if (one) {
                    const float wa = x ? w_other : w, wb = x ? w : w_other;  // of O0, of O1
                    uint32_t o1[32];
                    tmem_ld32(t_lane + 256u + D + c * 32, o1);
                    tmem_ld_wait();
                    reg_fence32(o1);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = f2u(other ? fmaf(wa, u2f(o[e]), wb * u2f(o1[e])) : wa * u2f(o[e]));
                }
                if (spoiled) {  // add the non-finite values of the edge tiles that this row sees
                    const __nv_bfloat16 *V = static_cast<const __nv_bfloat16 *>(a.v) + static_cast<size_t>(r.bk) * a.Skv * D + c * 32;
                    const int end = min(r.L, (r.j0 + r.n) * kN);
#pragma unroll 1
                    for (int key = (r.j0 + edge) * kN; key < end; ++key) {
                        if (!(visible32(set, key - r.past) & 1u)) continue;
                        const uint32_t *vr = reinterpret_cast<const uint32_t *>(V + static_cast<size_t>(key) * D);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint32_t v = vr[e], nf = nonfinite2(v);
                            if (nf & 0xffffu) o[2 * e] = f2u(u2f(o[2 * e]) + bf16lo_to_f32(v));
                            if (nf & 0xffff0000u) o[2 * e + 1] = f2u(u2f(o[2 * e + 1]) + bf16hi_to_f32(v));
                        }
                    }
                }
                if (write && r.slot >= 0) {
                    // four columns of all the slot's rows side by side: a warp writes 512 bytes at once
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o) + (static_cast<size_t>(r.slot) * (D / 4) + c * 8) * slot_rows + slot_row;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e * slot_rows] = make_float4(u2f(o[4 * e]), u2f(o[4 * e + 1]), u2f(o[4 * e + 2]), u2f(o[4 * e + 3]));
                } else if (write) {
                    uint4 *dst = reinterpret_cast<uint4 *>(out + c * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t pk[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            pk[y] = live ? pack_bf16x2(u2f(o[8 * e + 2 * y]) * inv, u2f(o[8 * e + 2 * y + 1]) * inv) : 0u;
                        dst[e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                }
            }
            if (write && r.slot >= 0 && (!one || x == 0))
                reinterpret_cast<float2 *>(a.part_ml)[static_cast<size_t>(r.slot) * slot_rows + slot_row] = make_float2(m, sum);
            mbar_arrive(&bars.run_empty[k % kRing]);
            tc_fence_before();
            __syncwarp();
            // both streams are done with each other's O and with ex
            if (one) join();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && bars.abort) report_timeout(a.status, 0x44);
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
// x and o hold the first ones already.
constexpr int kAhead = 4;
template <int C, bool Early, typename T, typename Part, typename Column>
__device__ __forceinline__ void merge_row(int n, bool live, T *out, Part part, Column column,
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
}

// bf16: block (i, y) merges 32 rows of the unit that begins in CTA i of the main
// kernel and ends in a later one: slot 2 i + 1, then slot 2 c of the CTAs after
// it.  Lane = row, as the partial results lie; warp = D / 8 columns.
// Early: the first slots are loaded beside the look-up, parts or not (of 2 n_split).
template <int D, bool Early>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeArgs a, const int slot_rows) {
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x, rr = blockIdx.y * 32 + threadIdx.x % 32, warp = threadIdx.x / 32;
    constexpr int C = D / 32;
    auto slot = [&](int c) { return static_cast<size_t>(c == 0 ? 2 * i + 1 : 2 * (i + c)); };
    auto part = [&](int c) { return reinterpret_cast<const float2 *>(a.part_ml)[slot(c) * slot_rows + rr]; };
    auto column = [&](int c, int e) {
        return reinterpret_cast<const float4 *>(a.part_o)[(slot(c) * (D / 4) + warp * C + e) * slot_rows + rr];
    };
    float2 x[kAhead];
    float4 o[kAhead][C];
    if (Early) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int c = min(y, a.n_split - 1 - i);
            x[y] = part(c);
#pragma unroll
            for (int e = 0; e < C; ++e) o[y][e] = column(c, e);
        }
    }
    const int4 rec = reinterpret_cast<const int4 *>(a.merge)[2 * i], rec2 = reinterpret_cast<const int4 *>(a.merge)[2 * i + 1];
    if (rec.x < 0) return;
    const int bk = rec.x, tile = rec.y, b = rec.z, last = rec.w, nd = rec2.x, past = rec2.y;
    const int G = a.H / a.H_kv, q = tile * kM + rr;
    if (q >= G * a.T) return;
    const int h = (bk - b * a.H_kv) * G + q / a.T, t = q % a.T;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + b * a.o_bs + h * a.o_hs + t * a.o_ts + warp * 4 * C;
    merge_row<C, Early>(last - i + 1, t < nd && past + t >= 0, out, part, column, x, o);
}

// fp32: one warp per row, n_split parts of `chunk` keys.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_f32_kernel(const TreeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int G = a.H / a.H_kv, rows = G * a.T, lane = threadIdx.x % 32;
    const long long R = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
    if (R >= static_cast<long long>(a.B) * a.H_kv * rows || lane >= D / 4) return;
    const int bk = static_cast<int>(R / rows), r = static_cast<int>(R % rows), b = bk / a.H_kv, g = bk % a.H_kv;
    const int t = r % a.T;
    const Draft d = draft_of(a, b);
    const bool live = t < d.n && d.past + t >= 0;
    float *out = static_cast<float *>(a.out) + b * a.o_bs + (g * G + r / a.T) * a.o_hs + t * a.o_ts + 4 * lane;
    float2 x[kAhead];
    float4 o[kAhead][1];
    merge_row<1, false>(live ? (d.L + a.chunk - 1) / a.chunk : 0, live, out,
                        [&](int c) { return reinterpret_cast<const float2 *>(a.part_ml)[R * a.n_split + c]; },
                        [&](int c, int) { return reinterpret_cast<const float4 *>(a.part_o)[(R * a.n_split + c) * (D / 4) + lane]; },
                        x, o);
}

// No cache rows at all: zeros.
__global__ void tree_zero_kernel(const TreeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const long long n = static_cast<long long>(a.B) * a.H * a.T * (a.D / 8);
    for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const long long r = i / (a.D / 8), c = i % (a.D / 8);
        const long long t = r % a.T, h = r / a.T % a.H, b = r / a.T / a.H;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + b * a.o_bs + h * a.o_hs + t * a.o_ts + c * 8) =
            make_uint4(0u, 0u, 0u, 0u);
    }
}

template <int D, bool Single>
cudaError_t launch_tree_t(const TreeArgs &a, int row_tiles, const CUtensorMap &tk, const CUtensorMap &tv) {
    using L = Layout<D, Single>;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, Single>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         L::kSmemBytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(a.n_split);
    e = launch_pdl(tree_tc_kernel<D, Single>, dim3(grid), dim3(kThreads), L::kSmemBytes, a.stream, a, row_tiles, tk, tv);
    if (e != cudaSuccess || grid == 1) return e;
    const int slot_rows = L::kQTiles * kM;
    const int rows = (a.H / a.H_kv) * a.T;
    const unsigned y = static_cast<unsigned>(((rows < slot_rows ? rows : slot_rows) + 31) / 32);
    // Early where units have several CTAs each (one sequence of 1500 rows 13.7 -> 12.8
    // us); where two share a unit now and then, loads for nothing and their registers
    // cost more (16 sequences 63.5 -> 64.5 us).
    const long long units = static_cast<long long>(a.B) * a.H_kv * ((row_tiles + L::kQTiles - 1) / L::kQTiles);
    return launch_pdl(grid >= 3 * units ? tree_join_kernel<D, true> : tree_join_kernel<D, false>, dim3(grid - 1, y),
                      dim3(256), 0, a.stream, a, slot_rows);
}

}  // namespace

int tree_tc_grid(int B, int H, int H_kv, int T, int Skv, int n_sm) {
    const int row_tiles = ((H / H_kv) * T + kM - 1) / kM;
    const long long tiles = Skv > kN ? (static_cast<long long>(Skv) + kN - 1) / kN : 1;
    const long long total = static_cast<long long>(B) * H_kv * ((row_tiles + 1) / 2) * (tiles + kUnitCost);
    if (total * 2 >= (1LL << 31)) return -1;  // the kernel counts in 32 bits
    const long long most = (total + kMinCost - 1) / kMinCost;
    return static_cast<int>(most < n_sm ? most : n_sm);
}

int tree_tc_slot_rows(int H, int H_kv, int T) { return (H / H_kv) * T <= kM ? kM : 2 * kM; }

cudaError_t launch_tree_zero(const TreeArgs &a) {
    return launch_pdl(tree_zero_kernel, dim3(static_cast<unsigned>(a.n_sm)), dim3(256), 0, a.stream, a);
}

cudaError_t launch_tree_tc(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv) {
    const int row_tiles = ((a.H / a.H_kv) * a.T + kM - 1) / kM;
    if (a.D == 64)
        return row_tiles == 1 ? launch_tree_t<64, true>(a, row_tiles, tk, tv) : launch_tree_t<64, false>(a, row_tiles, tk, tv);
    return row_tiles == 1 ? launch_tree_t<128, true>(a, row_tiles, tk, tv) : launch_tree_t<128, false>(a, row_tiles, tk, tv);
}

cudaError_t launch_tree_merge_f32(const TreeArgs &a) {
    const long long R = static_cast<long long>(a.B) * a.H * a.T;
    const dim3 grid(static_cast<unsigned>((R + 7) / 8));
    return a.D == 64 ? launch_pdl(tree_merge_f32_kernel<64>, grid, dim3(256), 0, a.stream, a)
                     : launch_pdl(tree_merge_f32_kernel<128>, grid, dim3(256), 0, a.stream, a);
}

}  // namespace attn
