// Attention of new tokens over a paged KV cache on the sm_103a tensor cores
// (attn_fwd_paged, bf16).
//
// Sequence s holds L tokens in pages of P rows, named by its row of the page table;
// the last n of them are new and have queries.  Token i of those sees the keys j <= L - n + i:
//     out_i = softmax over visible j of (scale q_i . k_j) times v_j.
// One form serves chunks of prompts, single tokens, and both in one call.
//
// Rows and units.  The G = H / H_kv query heads of a cached head and kTok = 128 / G
// tokens are the rows of a 128-row tile, token by token (row r: token r / G, head
// r % G), as one TMA box of (64 columns, G heads, kTok tokens) leaves them; groups of
// more than 128 heads are cut.  A unit is a cached head of a sequence with two row tiles
// (one, where the sequence has no more tokens).  It reads every key once for up to 256
// rows; on the diagonal it wastes 2 kTok keys at most, as heads, not tokens, fill the tile.
//
// Work split.  All units lie end to end on an axis of keys: unit u of a sequence takes
// max(L - n, 0) + 127 + (u + 1) 2 kTok keys and kUnitCost tiles for its start and end, so
// that the place of a unit is a quadratic in u and no list is needed.  CTA i of N takes
// the tiles that begin in the i-th equal part of the axis: no tail whatever the lengths
// are, and at most two units a CTA are shared with neighbours.  Those leave unnormalised
// O, running max and sum in fp32 in the CTA's slots of the workspace, for a merge in
// the order of the keys; whole units are written out directly.
//
// Few units of one row tile (up to an SM each) are clusters of one to eight CTAs instead, with
// equal parts of the unit's tiles, which meet in distributed shared memory: no axis, no
// workspace, no second kernel.
//
// Pages.  A 128-key tile is copied by boxes that lie in one page each (rows: the largest
// power of two up to 128 that divides P), each lane of the loading warp with its own box
// and its own entry of the table, fetched a tile ahead.  Boxes past the last visible key are not
// copied; an entry that is no page reads as zeros (TMA's fill).  What a small box costs is
// its instruction (some 25 ns each, one after the other), so one box brings all D columns: in
// shared memory a tile is groups of 8 rows, in each the 64-column blocks of 8 x 128 bytes
// one behind the other, which a view of (64 columns, 8 rows, D / 64 blocks, groups of
// rows, heads of pages) writes and the strides of the MMA's descriptors take.  Where
// the heads of all pages are not evenly spaced, boxes are the blocks themselves.
//
// Two softmax warpgroups (streams) keep two S and two O accumulators in TMEM busy.  A
// unit with two row tiles gives each stream one of them, and both read the same K/V
// tiles.  A unit with one gives the streams alternate K/V tiles; they join at its end:
//     two tiles:  S0_0 S1_0 | PV0_j S0_{j+1} PV1_j S1_{j+1} | ...
//     one tile:   S0_0 S1_1 | PV_j S_{j+2} (stream j & 1)   | ...
//
// A weight of zero does not hide an infinite or NaN value from the second product
// (0 * inf), and a page's rows past the sequence's end hold whatever they were left with,
// so two guard warps pass over the V of the tiles that some row sees a part of (edge
// tiles): rows past the unit's last key become zeros, non-finite elements become zeros
// which the epilogue adds back to the rows that see them.
//
// Measured (H 32 / 8, D 128):
//   64 sequences of up to 8192 keys in pages of 64, one token each, 1.29 GB     196 us, 6.6 TB/s
//   16 of up to 4096, all 32 heads cached, pages of 16, 0.56 GB                 100 us, 5.6 TB/s
//   60 of up to 6000 and chunks of 512, 512, 300 and 77 tokens, pages of 32     150 us
//   4096 tokens, the last of 32768, 2.06 TFLOP    1.19 ms, 1730 TFLOP/s (1.4 ms at the power limit)
//   one sequence of 1501 keys (table of up to 10600 tokens; 13.7 in a wider one)  9.1 us
//   256 of 100 to 1000 keys, pages of 16, 0.59 GB                               179 us, 3.3 TB/s
// The first is bound by HBM (a plain copy runs at 6.8 TB/s).  The second by the loading warp: a
// tile of eight boxes takes it some 1250 cycles (175 and 58 a box in the copies, the rest in
// waiting, announcing and looking up), at which all SMs just draw 7.2 TB/s.  The third by both
// that (four boxes) and the units' ends, where loads in flight drain; the fourth by the chain S,
// softmax, P V; the fifth by latency; the last by the units' ends (four tiles a unit).
// Other forms, in the first, second, third and fifth: loads of one 64-column block each 209, 154,
// 210 and 16.8 us; a loading loop for each form of unit 177 us in the third; every tile
// masked, for the sake of lanes without a row, 199, 104, 161 us; what a load needs computed behind
// its wait 3 us more in the third, 9.5 us in the fifth; few rows spread over all lanes (a row's columns
// over the warps), which halves the softmax of a tile but adds 1 us to the end of a unit, 3 us
// less, 11 us more and 1 us more in the first, third and fifth.
//
// Roles (12 warps): warp 3 walks the CTA's run and loads Q, K_j, V_j, warp 2 allocates
// TMEM and issues the MMAs, warps 0-1 guard, warps 4-7 and 8-11 are the streams (thread =
// row = TMEM lane); a warp none of whose rows sees a key only keeps step.
#include "clusters.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "serving.cuh"

#include <climits>
#include <type_traits>

namespace attn {
namespace {

constexpr int kN = 128;          // keys per K/V tile
constexpr int kM = 128;          // rows per tile
constexpr int kThreads = 384;
// Warps w, w + 4 and w + 8 share a scheduler.  A few rows keep only warps 4 and 8 busy, so the
// warps on which they wait lie elsewhere (loads by warp 0, MMAs by warp 1: one user 10.1 against
// 9.7 us, all heads 101 against 100).
constexpr int kLoadWarp = 3, kMmaWarp = 2;
// Registers after setmaxnreg: 128 * 80 + 256 * 208 <= 384 * 168.  The loading warp spills below
// 80, the softmax below 208 (96 and 200: 177 us for the third case above).
constexpr uint32_t kRegsOther = 80;     // warps 0-3
constexpr uint32_t kRegsSoftmax = 208;  // warps 4-11
constexpr int kTmemCols = 512;   // S0 0, S1 128, O0 256, O1 256 + D
constexpr int kRing = 4;         // unit runs in flight between the roles
constexpr int kRingReaders = 32 + 256;
constexpr int kGuardRing = 16;   // an edge tile holds a K/V stage: fewer than 16 at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kHugeLog2 = 16777216.0f;  // 2^24
// The axis, with what other values cost in the first three cases above.
constexpr int kUnitCost = 5;   // what a unit costs beside its tiles, in tiles (4: 199, 100, 152; 7: 197, 103, 152 us)
constexpr int kMinTiles = 2;   // fewest tiles' worth of keys a CTA takes (4: 128 tokens over 500 keys 18.9 against 17.9 us)
constexpr int kWeightTwo = 6;  // quarters of a tile's cost, where a unit has two row tiles (7: 157 us in the third; 4 and 5: worse by
                               // 30 and 8 us in an earlier form)
// The longest axis: the host accepts no call whose axis could be longer.  Offsets that are none (decreasing: sequences
// overlap) can make it longer all the same; it is no work then, before a place on it times the number of CTAs wraps.
constexpr long long kMaxAxis = 1ll << 52;
static_assert(4 * kMinTiles >= kWeightTwo, "a tile begins in every share: the merge reads all CTAs from a unit's first to its last");

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// 5-D: the first three coordinates 0.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c3), "r"(c4)
        : "memory");
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ long long prefix(long long v, int lane) {
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    return v;
}

// One sequence: first token, new tokens, keys.
struct Seq {
    int c0, n, L;
};

__device__ __forceinline__ Seq seq_of(const PagedArgs &a, int s) {
    Seq q;
    int c1;
    if (a.cu_seqlens) {
        q.c0 = min(max(a.cu_seqlens[s], 0), a.T);
        c1 = min(max(a.cu_seqlens[s + 1], q.c0), a.T);
    } else {
        q.c0 = s * a.per_seq;
        c1 = q.c0 + a.per_seq;
    }
    q.n = c1 - q.c0;
    q.L = a.cache_len ? min(max(a.cache_len[s], 0), a.max_len) : a.max_len;
    return q;
}

// a / b, in 32 bits where they do (a 64-bit division is a call of some 100 instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

// The units of one cached head (and group of heads) of a sequence on the axis: unit u of nu
// takes [at(u), at(u + 1)), its tile j begins at at(u) + j tile.
struct Units {
    int nu, step;   // units, tokens of a unit
    int weight;     // quarters a key
    int tile;       // quarters a K/V tile
    long long base;
    __device__ __forceinline__ Units(const Seq &q, int tokens, int one_tile) {
        nu = (q.n + tokens - 1) / tokens;
        step = min(tokens, q.n);
        const bool two = q.n > one_tile;
        weight = two ? kWeightTwo : 4;
        tile = weight * kN;
        base = static_cast<long long>(weight) * (max(q.L - q.n, 0) + kN - 1) + kUnitCost * kN * 4;
    }
    __device__ __forceinline__ long long at(int u) const {
        return u * base + static_cast<long long>(u) * (u + 1) / 2 * (step * weight);
    }
    // The first of a unit's nt tiles that lies behind a cut at x, counted from the unit's begin.
    __device__ __forceinline__ int cut(long long x, int nt) const {
        if (x >= static_cast<long long>(nt) * tile) return nt;
        return x <= 0 ? 0 : static_cast<int>(quotient(x + tile - 1, tile));
    }
};

// A run of K/V tiles [j0, j0 + n) of one unit.
struct Run {
    int seq, hs;    // sequence, cached head * groups of heads + group
    int tok0, left; // first token of the unit in the sequence, tokens from there on
    int j0, n;      // n < 0: no more work
    int slot;       // workspace slot, -1: the whole unit, written out
    int keys;       // keys that the unit's last row sees
    int past;       // keys in front of the sequence's first new token (may be negative)
    int c0;         // first token of the sequence
};

struct GuardReq {
    int stage;   // K/V stage of an edge tile, kEnd: no more work
    int parity;  // of the stage's kv_full
    int rows;    // rows of the tile that the unit sees
    int run;     // ring slot
};
constexpr int kEnd = -1;
constexpr int kNoBox = -1;    // the row of a box that is not copied
constexpr int kBadPage = -1;  // out of range in every view of the pages

// Single: every unit has one row tile; its second Q buffer is one more K/V stage.
template <int D, bool Single>
struct Layout {
    static constexpr int kSub = D / 64;
    static constexpr int kBlock = 128 * 128;        // 128 rows x 128 bytes
    static constexpr int kTile = kSub * kBlock;
    static constexpr int kQTiles = Single ? 1 : 2;
    static constexpr int kStages = D == 128 ? (Single ? 5 : 4) : 8;
    static constexpr int kRingOff = kQTiles * kTile;
    static constexpr int kExOff = kRingOff + kStages * kTile;
    static constexpr int kStageOff = kExOff + 256 * 8;   // per softmax warp: 32 rows x 64 bytes of output
    static constexpr int kBarOff = kStageOff + 8 * 2048;
    static constexpr int kSmemBytes = kBarOff + 1024 + 1024;
};

struct Bars {
    uint64_t q_full;            // Q of run k staged: phase k
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

__device__ __forceinline__ Run read_run(Bars &bars, int slot) {
    const volatile Run &s = bars.run[slot];
    return Run{s.seq, s.hs, s.tok0, s.left, s.j0, s.n, s.slot, s.keys, s.past, s.c0};
}
__device__ __forceinline__ bool take_run(Bars &bars, int k, Run *r) {
    if (!mbar_wait_warp(&bars.run_full[k % kRing], (k / kRing) & 1, &bars.abort)) return false;
    *r = read_run(bars, k % kRing);
    return true;
}

// First edge tile of a run, relative to j0: a tile that some row sees only a part of.
__device__ __forceinline__ int edge_of(const Run &r) { return min(r.n, max(0, max(0, r.past + r.tok0 + 1) / kN - r.j0)); }
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + kN - 1) / kN); }

// Row r of row tile x of a run: its token in the sequence, its query head, whether it
// exists, and the keys [0, lim) it sees.
struct Row {
    int token, head, lim;
    bool valid;
};
__device__ __forceinline__ Row row_of(const PagedArgs &a, int hs, int tok0, int left, int past, int x, int r) {
    const int t = r / a.heads, g = r - t * a.heads + (hs % a.groups) * a.heads, i = x * a.tokens + t, G = a.H / a.H_kv;
    Row w;
    w.valid = t < a.tokens && i < left && g < G;
    w.token = tok0 + i;
    w.head = hs / a.groups * G + g;
    w.lim = w.valid ? max(0, past + w.token + 1) : 0;
    return w;
}

// A cluster's CTA leaves its part of its rows in its K/V ring: O, D + 4 floats a row, then max
// and sum.
template <int D>
__device__ __forceinline__ float2 *cluster_ml(uint8_t *ring) {
    return reinterpret_cast<float2 *>(ring + kM * (D + 4) * 4);
}

// Adds to columns [c, c + 32) of a row the non-finite values that the guard took out of the
// run's edge tiles, of the keys that the row sees.
__device__ __forceinline__ void add_nonfinite(const PagedArgs &a, const Run &r, int lim, int c, uint32_t (&o)[32]) {
    const int end = min(lim, (r.j0 + r.n) * kN);
    const int32_t *table = a.page_table + static_cast<long long>(r.seq) * a.table_stride;
#pragma unroll 1
    for (int key = (r.j0 + edge_of(r)) * kN; key < end; ++key) {
        const int entry = page_of_key(a, key), page = table[entry];
        if (!is_page(a, page)) continue;
        const uint32_t *vr = reinterpret_cast<const uint32_t *>(
            static_cast<const __nv_bfloat16 *>(a.v) + page * a.v_ps + (r.hs / a.groups) * a.v_hs + (key - entry * a.P) * a.v_rs + c);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t v = vr[e], nf = nonfinite2(v);
            if (nf & 0xffffu) o[2 * e] = f2u(u2f(o[2 * e]) + bf16lo_to_f32(v));
            if (nf & 0xffff0000u) o[2 * e + 1] = f2u(u2f(o[2 * e + 1]) + bf16hi_to_f32(v));
        }
    }
}

template <int D, bool Single, bool Cluster>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv) {
    using L = Layout<D, Single>;
    static_assert(!Cluster || Single, "a cluster has one row tile");
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + L::kRingOff;
    float2 *ex = reinterpret_cast<float2 *>(smem + L::kExOff);  // [stream][row] max, sum
    Bars &bars = *reinterpret_cast<Bars *>(smem + L::kBarOff);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        mbar_init(&bars.q_full, 1);
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
    if (warp == kMmaWarp) {
        tmem_alloc(&bars.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // rows that no load of Q writes have scores of 0: their lanes never take a rare path
    for (int i = threadIdx.x; i < L::kQTiles * L::kTile / 16; i += kThreads) st_shared_v4(smem_u32(smem) + i * 16, 0u, 0u, 0u, 0u);
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    griddep_launch_dependents();
    griddep_wait();

    if (warp == kLoadWarp) {
        // ================================================================ walk and TMA loads
        regs_dec<kRegsOther>();
        const int per = a.H_kv * a.groups;  // heads, or groups of them, of a sequence
        const int tokens = (Single ? 1 : 2) * a.tokens;  // of a unit
        auto cost_of = [&](const Seq &q) {
            const Units u(q, tokens, a.tokens);
            return u.at(u.nu) * per;
        };
        // A cluster's CTAs share the tiles of its one unit; else CTA I of N takes what begins in
        // [total I / N, total (I + 1) / N) of the axis (whose length the host has checked).
        long long total = 0, lo = 0, hi = 0, base = 0;  // base: first position of sequence b's units
        int N = 1, b = 0;
        bool idle = false;
        Seq q{0, 0, 0};
        if (Cluster) {
            b = static_cast<int>(blockIdx.x >> a.cluster_shift) / per;
            q = seq_of(a, b);
            idle = q.n == 0;
            hi = LLONG_MAX;
        } else {
            Seq mine{0, 0, 0};  // sequence b0 + lane
            long long t = 0, sum = 0;
            for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
                mine = seq_of(a, min(b0 + lane, a.n_seq - 1));
                t = b0 + lane < a.n_seq ? cost_of(mine) : 0;
                total = min(total + t, kMaxAxis + 1);
            }
            if (a.n_seq <= 32) {
                sum = prefix(t, lane);
                total = __shfl_sync(0xffffffffu, sum, 31);
            } else {
#pragma unroll 1
                for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
            }
            const long long most = total / (4 * kN * kMinTiles);
            N = static_cast<int>(min(max(most, 1ll), static_cast<long long>(gridDim.x)));
            const int I = blockIdx.x;
            idle = I >= N || total == 0 || total > kMaxAxis;
            const long long each = quotient(total, N);
            const int odd = static_cast<int>(total - each * N);
            if (!idle) lo = each * I + odd * I / N, hi = each * (I + 1) + odd * (I + 1) / N;
            for (int b0 = 0; !idle && b0 < a.n_seq; b0 += 32) {  // the sequence that holds position lo
                if (a.n_seq > 32) {
                    mine = seq_of(a, min(b0 + lane, a.n_seq - 1));
                    t = b0 + lane < a.n_seq ? cost_of(mine) : 0;
                    sum = prefix(t, lane);
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
            q = Seq{__shfl_sync(0xffffffffu, mine.c0, b % 32), __shfl_sync(0xffffffffu, mine.n, b % 32),
                    __shfl_sync(0xffffffffu, mine.L, b % 32)};
        }
        Units units(q, tokens, a.tokens);
        int hs = 0, u = 0, j = 0;
        long long pos = base;  // of unit u of hs
        auto keys_of = [&](int unit) { return max(0, min(q.L, q.L - q.n + min((unit + 1) * tokens, q.n))); };
        auto next_unit = [&] {
            pos += units.at(u + 1) - units.at(u);
            j = 0;
            if (++u < units.nu) return;
            u = 0;
            if (++hs < per) return;
            hs = 0;
            while (++b < a.n_seq) {
                q = seq_of(a, b);
                if (q.n > 0) {
                    units = Units(q, tokens, a.tokens);
                    break;
                }
            }
        };
        if (Cluster) {
            hs = static_cast<int>(blockIdx.x >> a.cluster_shift) - b * per;
            j = tiles_of(keys_of(0)) * static_cast<int>(cluster_rank()) >> a.cluster_shift;
        } else if (!idle) {
            const long long one = units.at(units.nu);
            hs = static_cast<int>(quotient(lo - base, one));
            pos += hs * one;
            int top = units.nu;  // at(u) <= lo - pos < at(top)
            while (top - u > 1) {
                const int mid = (u + top) / 2;
                if (units.at(mid) <= lo - pos)
                    u = mid;
                else
                    top = mid;
            }
            pos += units.at(u);
            const int nt = tiles_of(keys_of(u));
            j = units.cut(lo - pos, nt);
            if (j == nt) next_unit();
        }
        // this lane's box of a tile: rows [i box, (i + 1) box), of the columns from 64 c on
        // where a box does not hold them all
        const int boxes = kN / a.box, i = lane % boxes, c = lane / boxes;
        const bool carries = lane < boxes * (a.halves ? L::kSub : 1);
        const uint32_t box_bytes = static_cast<uint32_t>(a.box * D * 2), box_at = i * box_bytes + c * 1024;
        const int page_inc = kN / a.P, row_inc = kN % a.P;  // from tile to tile
        int issued = 0, stage = 0, requests = 0, k = 0, q_loads = 0;
        uint32_t stage_phase = 1;  // of kv_empty: the first round of the ring waits for nothing
        bool ok = true;
        int4 *record = reinterpret_cast<int4 *>(a.merge) + 2 * blockIdx.x;  // of the unit shared with later CTAs
        if (!Cluster && lane == 0) record[0] = make_int4(-1, 0, 0, 0);
        while (ok) {
            const int slot = k % kRing;
            if (k >= kRing && !(ok = mbar_wait_warp(&bars.run_empty[slot], ((k / kRing) - 1) & 1, &bars.abort))) break;
            Run r{0, 0, 0, 0, 0, -1, 0, 0, 0, 0};
            int nt = 0;
            if (!idle && b < a.n_seq && pos < hi) {  // r.n = 0: a CTA of a cluster without a tile
                const int keys = keys_of(u);
                nt = tiles_of(keys);
                const int end = Cluster ? nt * static_cast<int>(cluster_rank() + 1) >> a.cluster_shift : units.cut(hi - pos, nt);
                if (Cluster || end > j) {
                    r.seq = b;
                    r.hs = hs;
                    r.tok0 = u * tokens;
                    r.left = q.n - r.tok0;
                    r.keys = keys;
                    r.past = q.L - q.n;
                    r.c0 = q.c0;
                    r.j0 = j;
                    r.n = end - j;
                    r.slot = Cluster || r.n == nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (j == 0 ? 1 : 0);
                    if (!Cluster && j == 0 && r.n < nt) {  // the unit begins here and goes on in CTAs up to the record's,
                                                           // the last that begins at or before its last tile
                        const long long last = pos + static_cast<long long>(nt - 1) * units.tile;
                        if (lane == 0) {
                            record[0] = make_int4(b, hs, r.tok0, static_cast<int>(quotient((last + 1) * N - 1, total)));
                            record[1] = make_int4(r.left, r.past, r.c0, 0);
                        }
                    }
                }
            }
            auto publish = [&] {
                if (lane == 0) {
                    volatile Run &w = bars.run[slot];
                    w.seq = r.seq, w.hs = r.hs, w.tok0 = r.tok0, w.left = r.left, w.j0 = r.j0, w.n = r.n, w.slot = r.slot;
                    w.keys = r.keys, w.past = r.past, w.c0 = r.c0;
                    *static_cast<volatile int *>(&bars.spoiled[slot]) = 0;
                    mbar_arrive(&bars.run_full[slot]);
                }
                __syncwarp();
            };
            if (r.n < 0) {
                publish();
                break;
            }
            const int edge = edge_of(r), head = r.hs / a.groups;
            // This lane's box of the next tile to be looked up: its key, its entry of the table and its row
            // in that page.
            const int k_head = head * a.k_hstep, v_head = head * a.v_hstep;
            int next_key = r.j0 * kN + i * a.box, next_row = page_of_key(a, next_key);
            const int32_t *next_entry = a.page_table + static_cast<long long>(r.seq) * a.table_stride + next_row;
            next_row = next_key - next_row * a.P;
            const int last_key = min(r.keys, (r.j0 + r.n) * kN);
            struct Box {
                int page, row;  // page: as it stands in the table, untouched until its tile is loaded (two tiles later)
            };
            auto look_up = [&] {
                Box x{kBadPage, kNoBox};
                if (carries && next_key < last_key) x.page = *next_entry, x.row = next_row;
                next_key += kN;
                next_entry += page_inc;
                next_row += row_inc;
                if (next_row >= a.P) next_row -= a.P, ++next_entry;
                return x;
            };
            auto load = [&](int jj, auto v, const Box &x) {  // K or V of tile jj into the next stage
                constexpr bool kv = decltype(v)::value;
                if (!ok) return;
                // before the wait: what does not depend on it
                const int inside = r.keys - (r.j0 + jj) * kN;
                const uint32_t bytes = inside >= kN ? kN * D * 2u : inside > 0 ? ((inside + a.box - 1) & -a.box) * (D * 2u) : 0u;
                const unsigned at = static_cast<unsigned>(x.page) * (kv ? a.v_pstep : a.k_pstep) + (kv ? v_head : k_head);
                const int entry = is_page(a, x.page) ? a.halves ? x.page : static_cast<int>(at) : kBadPage;
                if (!__all_sync(0xffffffffu, mbar_try_wait(&bars.kv_empty[stage], stage_phase)) &&
                    !(ok = mbar_wait_warp(&bars.kv_empty[stage], stage_phase, &bars.abort)))
                    return;
                uint64_t *full = &bars.kv_full[stage];
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                uint8_t *dst = ring + stage * L::kTile;
                const CUtensorMap *map = kv ? &tv : &tk;
                if (x.row != kNoBox) {
                    if (a.halves)
                        tma_load_4d(dst + box_at, map, full, c * 64, x.row, head, entry);
                    else
                        tma_load_5d(dst + box_at, map, full, x.row / 8, entry);
                }
                if (kv && jj >= edge) {
                    if (lane == 0) {
                        volatile GuardReq &g = bars.req[requests % kGuardRing];
                        g.stage = stage, g.parity = stage_phase ^ 1, g.rows = inside, g.run = slot;
                        mbar_arrive(&bars.guard_full[requests % kGuardRing]);
                    }
                    ++requests;
                }
                ++issued;
                if (++stage == kStages) stage = 0, stage_phase ^= 1;
            };
            auto load_q = [&](int tiles) {  // once the last run's last S MMA has read the buffers
                if (r.n == 0) return;
                if (!ok || (k > 0 && !(ok = mbar_wait_warp(&bars.q_free, (k - 1) & 1, &bars.abort)))) return;
                if (lane == 0) {
                    const int h0 = head * (a.H / a.H_kv) + r.hs % a.groups * a.heads;
                    mbar_arrive_expect_tx(&bars.q_full, static_cast<uint32_t>(tiles * a.box_tokens * a.heads * D * 2));
                    for (int x = 0; x < tiles; ++x)
#pragma unroll
                        for (int cc = 0; cc < L::kSub; ++cc)
                            tma_load_3d(smem + x * L::kTile + cc * L::kBlock, &tq, &bars.q_full, cc * 64, h0,
                                        r.c0 + r.tok0 + x * a.tokens);
                }
                __syncwarp();
                ++q_loads;
            };
            const bool one = Single || r.left <= a.tokens;
            const int lead = one ? 2 : 1;  // tiles that K is ahead: K0 K1 | V0 K2 | V1 K3 or K0 | V0 K1 | V1 K2
            // boxes of tiles jj + lead - 2 to jj + lead + 1
            Box v2{kBadPage, kNoBox}, v1 = v2, now = look_up(), next = look_up();
            publish();
            if (k == 0) load_q(one ? 1 : 2);  // before the first K; later behind it
            for (int jj = -lead; jj < r.n && ok; ++jj) {
                if (jj == 0 && k > 0) load_q(one ? 1 : 2);
                if (jj >= 0) load(jj, std::true_type{}, one ? v2 : v1);
                if (jj + lead < r.n) load(jj + lead, std::false_type{}, now);
                v2 = v1, v1 = now, now = next, next = look_up();
            }
            ++k;
            if (Cluster) {
                b = a.n_seq;
                continue;
            }
            j += r.n;
            if (j == nt) next_unit();
        }
        if (lane == 0) {
            if (ok) {  // no more work for the guard
                *static_cast<volatile int *>(&bars.req[requests % kGuardRing].stage) = kEnd;
                mbar_arrive(&bars.guard_full[requests % kGuardRing]);
            }
            // never leave with copies still landing in shared memory
            volatile int never = 0;
            if (q_loads > 0) mbar_wait(&bars.q_full, (q_loads - 1) & 1, &never);
            for (int x = max(0, issued - kStages); x < issued; ++x)
                mbar_wait(&bars.kv_full[x % kStages], (x / kStages) & 1, &never);
        }
        __syncwarp();
        if (Cluster) cluster_sync(), cluster_sync();
    } else if (warp == kMmaWarp) {
        // ================================================================ MMA issuer
        regs_dec<kRegsOther>();
        const uint32_t idesc_s = idesc_bf16_f32(kM, kN, 0);
        const uint32_t idesc_o = idesc_bf16_f32(kM, D, 1);
        const uint64_t dq0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(ring), 16, L::kSub * 1024);
        const uint64_t dv0 = sdesc_sw128(smem_u32(ring), 1024, L::kSub * 1024);
        auto issue_s = [&](int x, int qbuf, int slot) {  // S_x = Q_qbuf K^T
            const uint64_t da = desc_add(dq0, (qbuf * L::kTile) >> 4), db = desc_add(dk0, (slot * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t q_off = ((kk / 4) * L::kBlock + (kk % 4) * 32) >> 4, k_off = ((kk / 4) * 1024 + (kk % 4) * 32) >> 4;
                mma_ss_warp(tmem + x * 128u, desc_add(da, q_off), desc_add(db, k_off), idesc_s, kk > 0);
            }
        };
        auto issue_pv = [&](int x, int slot, bool acc) {  // O_x (+)= P_x V
            const uint64_t db = desc_add(dv0, (slot * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
                mma_ts_warp(tmem + 256u + x * static_cast<uint32_t>(D), tmem + x * 128u + kk * 8,
                            desc_add(db, (kk * 16 * D * 2) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u);
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
            if (Cluster && n == 0) continue;
            const int edge = __shfl_sync(0xffffffffu, edge_of(r), 0);
            const bool one = Single || __shfl_sync(0xffffffffu, r.left, 0) <= a.tokens;
            if (!(ok = mbar_wait_warp(&bars.q_full, k & 1, &bars.abort))) break;
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
        if (Cluster) cluster_sync(), cluster_sync();
    } else if (warp < 4) {
        // ================================================================ guard of the edge V tiles
        regs_dec<kRegsOther>();
        const int tid = threadIdx.x;
        for (int q = 0;; ++q) {
            const int slot = q % kGuardRing;
            // a request comes after its load was issued, and its stage is not reused
            // before guard_clean: kv_full cannot be a phase off
            if (!mbar_wait_warp<64>(&bars.guard_full[slot], (q / kGuardRing) & 1, &bars.abort)) break;
            const volatile GuardReq &rq = bars.req[slot];
            const int stage = rq.stage, parity = rq.parity, inside = rq.rows, run = rq.run;
            if (stage < 0) break;
            if (!mbar_wait_warp(&bars.kv_full[stage], parity, &bars.abort)) break;
            const uint32_t tile = smem_u32(ring + stage * L::kTile);
            const bool bad = clean_v_tile<L::kSub, kN, 64, true>(tile, inside, tid);
            if (bad) *static_cast<volatile int *>(&bars.spoiled[run]) = 1;
            if (inside < kN || __any_sync(0xffffffffu, bad)) fence_proxy_async_shared();  // written: the MMA must see it
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.guard_clean[slot]);
        }
        __syncwarp();
        if (Cluster) cluster_sync(), cluster_sync();
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
            bool one;
            int n, lim;  // tiles of this stream; this row sees columns [0, lim) from the run's first key on
            {
                Run r;
                if (!(ok = take_run(bars, k, &r))) break;
                if (r.n < 0) break;
                one = Single || r.left <= a.tokens;
                n = one ? (r.n - x + 1) / 2 : r.n;
                const Row w = row_of(a, r.hs, r.tok0, r.left, r.past, one ? 0 : x, row);
                const int most = __reduce_max_sync(0xffffffffu, w.lim);
                // a lane without a row hides no keys, so that only the edge tiles are masked
                lim = (w.valid ? w.lim : most) - r.j0 * kN;
                if (most <= 0) lim = INT_MIN;  // the whole warp only keeps step
            }
            float m_run = -INFINITY, l = 0.f;
            bool huge = sl2 == 0.f;  // some row of the warp is
            for (int i = 0; i < n; ++i) {
                const int j = one ? 2 * i + x : i;
                if (!(ok = mbar_wait_warp<32>(&bars.s_full[x], sp, &bars.abort))) break;
                sp ^= 1;
                if (lim == INT_MIN) {
                    mbar_arrive(&bars.p_ready[x]);
                    continue;
                }
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, s + c * 32);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_fence32(s + c * 32);
                const int t = lim - j * kN;  // this row sees columns [0, t)
                const bool masked = __any_sync(0xffffffffu, t < kN);
                if (masked) {  // 32 columns at a time: bits of those that the row sees
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int left = t - 32 * c;
                        const uint32_t see = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
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
                        const float first = mine ? sl2 : 1.f;
#pragma unroll
                        for (int e = 0; e < kN; ++e) s[e] = e < t ? f2u(__fmul_rn(u2f(s[e]), first)) : f2u(-INFINITY);
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
            const Row w = row_of(a, r.hs, r.tok0, r.left, r.past, one ? 0 : x, row);
            const bool live = w.lim > 0;
            const bool other = one && r.n > 1;  // the other stream has a part of the same rows
            float wt = 1.f, wt_other = 0.f, m = m_run, sum = l;
            if (one) {
                ex[x * kM + row] = make_float2(m_run, l);
                join();
                const float2 y = ex[(x ^ 1) * kM + row];
                m = fmaxf(m_run, y.x);
                const float ref = m == -INFINITY ? 0.f : m;
                wt = ex2_approx(m_run - ref);
                wt_other = ex2_approx(y.x - ref);
                sum = l * wt + y.y * wt_other;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const bool used = one ? y < r.n : true;
                if (used && (one || y == x) && ok) ok = mbar_wait_warp(&bars.o_full[y], o_uses[y] & 1, &bars.abort);
                if (used) ++o_uses[y];
            }
            tc_fence_after();
            if (Cluster) {
                // this CTA's part of its rows, for the cluster: the ring is free, every MMA on it is complete
                float *part = reinterpret_cast<float *>(ring) + row * (D + 4);
                if (__any_sync(0xffffffffu, w.valid)) {
#pragma unroll
                    for (int c = x * (D / 64), y = 0; y < D / 64; ++c, ++y) {
                        uint32_t o[32], o1[32];
                        tmem_ld32(t_lane + 256u + c * 32, o);
                        tmem_ld32(t_lane + 256u + D + c * 32, o1);
                        tmem_ld_wait();
                        reg_fence32(o);
                        reg_fence32(o1);
                        const float wa = x ? wt_other : wt, wb = x ? wt : wt_other;  // of O0, of O1
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = r.n == 0 || !live ? 0u : f2u(other ? fmaf(wa, u2f(o[e]), wb * u2f(o1[e])) : wa * u2f(o[e]));
                        if (*static_cast<volatile int *>(&bars.spoiled[k % kRing]) != 0 && live)
                            add_nonfinite(a, r, w.lim, c * 32, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(part + c * 32 + 4 * e) =
                                make_float4(u2f(o[4 * e]), u2f(o[4 * e + 1]), u2f(o[4 * e + 2]), u2f(o[4 * e + 3]));
                    }
                }
                if (x == 0) cluster_ml<D>(ring)[row] = make_float2(m, sum);  // both streams hold the same
                mbar_arrive(&bars.run_empty[k % kRing]);
                tc_fence_before();
                continue;
            }
            const bool write = ok && w.valid;
            const bool spoiled = *static_cast<volatile int *>(&bars.spoiled[k % kRing]) != 0 && live;
            const float inv = 1.f / sum;
            const int slot_row = (one ? 0 : x * kM) + row;
            // a unit of one row tile: stream 0 writes the first half of the columns, stream 1 the second
            const int c0 = one ? x * (D / 64) : 0, c1 = one ? c0 + D / 64 : D / 32;
            const long long token = static_cast<long long>(r.c0) + w.token;
            if (__any_sync(0xffffffffu, w.valid)) {
                // rows that the lanes store: 8 y + lane / 4, 16 bytes each
                const uint32_t stage = smem_u32(smem + L::kStageOff + (warp - 4) * 2048);
                const unsigned long long out = write && r.slot < 0
                    ? reinterpret_cast<unsigned long long>(static_cast<__nv_bfloat16 *>(a.out) + token * a.o_ts + w.head * a.o_hs) : 0ull;
                unsigned long long to[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) to[y] = __shfl_sync(0xffffffffu, out, 8 * y + lane / 4);
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    __syncwarp();
                    uint32_t o[32];  // TMEM of this CTA: loaded unconditionally, used only when valid
                    tmem_ld32((one ? t_lane + 256u : t_o) + c * 32, o);
                    tmem_ld_wait();
                    reg_fence32(o);
                    if (one) {
                        const float wa = x ? wt_other : wt, wb = x ? wt : wt_other;  // of O0, of O1
                        uint32_t o1[32];
                        tmem_ld32(t_lane + 256u + D + c * 32, o1);
                        tmem_ld_wait();
                        reg_fence32(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = f2u(other ? fmaf(wa, u2f(o[e]), wb * u2f(o1[e])) : wa * u2f(o[e]));
                    }
                    if (spoiled) add_nonfinite(a, r, w.lim, c * 32, o);
                    if (write && r.slot >= 0) {
                        // four columns of all the slot's rows side by side: a warp writes 512 bytes at once
                        float4 *dst = reinterpret_cast<float4 *>(a.part_o) +
                                      (static_cast<size_t>(r.slot) * (D / 4) + c * 8) * a.slot_rows + slot_row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e * a.slot_rows] = make_float4(u2f(o[4 * e]), u2f(o[4 * e + 1]), u2f(o[4 * e + 2]), u2f(o[4 * e + 3]));
                    }
                    if (r.slot < 0) {
                        // through the warp's buffer, so that a store writes 64 bytes of each of 8 rows
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t pk[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                pk[y] = live ? pack_bf16x2(u2f(o[8 * e + 2 * y]) * inv, u2f(o[8 * e + 2 * y + 1]) * inv) : 0u;
                            st_shared_v4(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), pk[0], pk[1], pk[2], pk[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int rr = 8 * y + lane / 4, q4 = lane % 4;
                            const uint4 v = ld_shared_v4(stage + rr * 64 + ((q4 ^ ((rr >> 1) & 3)) << 4));
                            if (to[y]) *reinterpret_cast<uint4 *>(to[y] + c * 64 + q4 * 16) = v;
                        }
                        __syncwarp();
                    }
                }
            }
            if (write && (!one || x == 0)) {
                if (r.slot >= 0)
                    reinterpret_cast<float2 *>(a.part_ml)[static_cast<size_t>(r.slot) * a.slot_rows + slot_row] = make_float2(m, sum);
                else if (a.lse)
                    a.lse[token * a.H + w.head] = live ? (m + log2f(sum)) * kLn2 : -INFINITY;
            }
            mbar_arrive(&bars.run_empty[k % kRing]);
            tc_fence_before();
            __syncwarp();
            // both streams are done with each other's O and with ex
            if (one) join();
        }
        if (Cluster) {
            // each CTA joins its share of the columns, the parts in the order of the keys
            __syncwarp();
            cluster_sync();
            const int n_cta = 1 << a.cluster_shift, quads = D / 4 >> a.cluster_shift;  // of a CTA's columns
            const Run r = read_run(bars, 0);
            const unsigned rank = cluster_rank();
#pragma unroll 1
            for (int i = static_cast<int>(threadIdx.x) - 128; i < (a.box_tokens * a.heads * (D / 4)) >> a.cluster_shift; i += 256) {
                const int rr = (i << a.cluster_shift) / (D / 4), c = (static_cast<int>(rank) * quads + (i & (quads - 1))) * 4;
                const Row w = row_of(a, r.hs, r.tok0, r.left, r.past, 0, rr);
                if (!w.valid) continue;
                float2 ml[kPagedCluster];
                float4 o[kPagedCluster];
                float M = -INFINITY, sum = 0.f;
                const float *part = reinterpret_cast<const float *>(ring) + rr * (D + 4) + c;
#pragma unroll
                for (unsigned y = 0; y < kPagedCluster; ++y) {
                    ml[y] = make_float2(-INFINITY, 0.f), o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (static_cast<int>(y) >= n_cta) continue;
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                                 : "=f"(ml[y].x), "=f"(ml[y].y) : "r"(map_rank(cluster_ml<D>(ring) + rr, y)));
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(o[y].x), "=f"(o[y].y), "=f"(o[y].z), "=f"(o[y].w) : "r"(map_rank(part, y)));
                }
#pragma unroll
                for (int y = 0; y < kPagedCluster; ++y) M = fmaxf(M, ml[y].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < kPagedCluster; ++y) {
                    const float f = ex2_approx(ml[y].x - ref);
                    sum = fmaf(f, ml[y].y, sum);
                    acc = make_float4(fmaf(f, o[y].x, acc.x), fmaf(f, o[y].y, acc.y), fmaf(f, o[y].z, acc.z), fmaf(f, o[y].w, acc.w));
                }
                const bool live = w.lim > 0;
                const float inv = 1.f / sum;
                const long long token = static_cast<long long>(r.c0) + w.token;
                store4(static_cast<__nv_bfloat16 *>(a.out) + token * a.o_ts + w.head * a.o_hs + c,
                       live ? make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
                if (a.lse && c == 0) a.lse[token * a.H + w.head] = live ? (M + log2f(sum)) * kLn2 : -INFINITY;
            }
            __syncwarp();
            cluster_sync();  // the parts have been read
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && bars.abort) report_timeout(a.status, 0x45);
}

// Block (i, y) merges 32 rows of the unit that begins in CTA i of the main kernel and
// ends in a later one: slot 2 i + 1, then slot 2 c of the CTAs after it.  Lane = row, as
// the partial results lie; warp = D / 8 columns.
// Early: the first slots are loaded beside the look-up, parts or not.
template <int D, bool Early>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x, rr = blockIdx.y * 32 + threadIdx.x % 32, warp = threadIdx.x / 32;
    constexpr int C = D / 32;
    auto slot = [&](int c) { return static_cast<size_t>(c == 0 ? 2 * i + 1 : 2 * (i + c)); };
    auto part = [&](int c) { return reinterpret_cast<const float2 *>(a.part_ml)[slot(c) * a.slot_rows + rr]; };
    auto column = [&](int c, int e) {
        return reinterpret_cast<const float4 *>(a.part_o)[(slot(c) * (D / 4) + warp * C + e) * a.slot_rows + rr];
    };
    float2 x[kAhead];
    float4 o[kAhead][C];
    if (Early) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int c = min(y, a.grid - 1 - i);
            x[y] = part(c);
#pragma unroll
            for (int e = 0; e < C; ++e) o[y][e] = column(c, e);
        }
    }
    const int4 rec = reinterpret_cast<const int4 *>(a.merge)[2 * i], rec2 = reinterpret_cast<const int4 *>(a.merge)[2 * i + 1];
    if (rec.x < 0) return;
    const Row w = row_of(a, rec.y, rec.z, rec2.x, rec2.y, rr / kM, rr % kM);
    if (!w.valid) return;
    const long long token = static_cast<long long>(rec2.z) + w.token;
    const bool live = w.lim > 0;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + token * a.o_ts + w.head * a.o_hs + warp * 4 * C;
    const float2 ml = merge_row<C, Early>(rec.w - i + 1, live, out, part, column, x, o);
    if (a.lse && warp == 0) a.lse[token * a.H + w.head] = live ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
}

template <int D, bool Single, bool Cluster>
cudaError_t launch_paged_t(const PagedArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv) {
    using L = Layout<D, Single>;
    const auto kernel = paged_tc_kernel<D, Single, Cluster>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(a.grid);
    e = launch_clusters(kernel, Cluster ? static_cast<unsigned>(a.cluster) : 1u, grid, kThreads, L::kSmemBytes, a.stream, a, tq, tk, tv);
    if (Cluster || e != cudaSuccess || grid == 1) return e;
    // Early where units have several CTAs each, as in tree_tc.cu
    const long long units = static_cast<long long>(a.n_seq) * a.H_kv * a.groups;
    return launch_pdl(Single && grid >= 3 * units ? paged_join_kernel<D, true> : paged_join_kernel<D, false>,
                      dim3(grid - 1, static_cast<unsigned>(a.slot_rows / 32)), dim3(256), 0, a.stream, a);
}

template <int D>
cudaError_t launch_paged_d(const PagedArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv) {
    return a.cluster ? launch_paged_t<D, true, true>(a, tq, tk, tv)
           : a.single ? launch_paged_t<D, true, false>(a, tq, tk, tv) : launch_paged_t<D, false, false>(a, tq, tk, tv);
}

}  // namespace

// Length of the axis of all units, at most.
double paged_tc_axis(const PagedArgs &a) {
    const double units = static_cast<double>(a.n_seq) + static_cast<double>(a.T) / a.tokens;
    return units * a.H_kv * a.groups * (kWeightTwo * (static_cast<double>(a.max_len) + a.T + kN) + 4 * kN * kUnitCost);
}

cudaError_t launch_paged_tc(const PagedArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv) {
    return a.D == 64 ? launch_paged_d<64>(a, tq, tk, tv) : launch_paged_d<128>(a, tq, tk, tv);
}

}  // namespace attn
