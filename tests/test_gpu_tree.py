"""GPU parity tests of attn_decode_tree against the definition in 64 bits; the
tolerances are derived in serving_ref.py."""
from __future__ import annotations

import math
import random

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import workloads as wl
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def tree(T, kind, seed):
    r = random.Random(seed)
    if kind == "chain":
        return [i - 1 for i in range(T)]
    if kind == "star":
        return [-1] * T
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(T)]
    return [-1 if i == 0 or r.random() < 0.15 else r.randint(0, i - 1) for i in range(T)]


def sight(parents, L, n):
    """(n, L) visibility of cache rows from the drafted tokens."""
    past = L - n
    see = torch.zeros(n, max(L, 0), dtype=torch.bool)
    see[:, :max(past, 0)] = True
    for t in range(n):
        j = t
        while 0 <= j:
            if past + j >= 0:
                see[t, past + j] = True
            p = parents[j]
            j = p if 0 <= p < j else -1
    for t in range(n):
        if past + t < 0:
            see[t] = False
    return see.cuda()


def verify(q, kc, vc, parents, lens, drafts, out, scale=None, only=None, what=""):
    B, H, T, D = q.shape
    G, Skv = H // kc.shape[1], kc.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        L = min(max(lens[b], 0), Skv) if lens is not None else Skv
        n = min(max(drafts[b], 0), T) if drafts is not None else T
        see = sight(parents[b], L, n)
        empty = ~see.any(1)
        assert torch.count_nonzero(out[b, :, n:]) == 0 and torch.count_nonzero(out[b, :, :n][:, empty]) == 0
        if n == 0 or bool(empty.all()):
            continue
        for h in range(H) if only is None else only:
            o, _, A, size = ref.attend(q[b, h, :n][~empty], kc[b, h // G, :L], vc[b, h // G, :L], see[~empty], scale)
            tol, _ = ref.bounds(q.dtype, D, L, scale, size, o, A)
            ref.check(out[b, h, :n][~empty], o, tol, f"{what} sequence {b} (L {L}, n {n}) head {h}")


def case(B, H, H_kv, T, Skv, D, lens, drafts, kind="random", dtype=BF16, seed=1, scale=None, only=None, one_tree=False):
    q = wl.random_tensors((B, T, H, D), seed, dtype=dtype, count=1)[0].transpose(1, 2)
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), seed + 1, dtype=dtype, count=2)
    parents = [tree(T, kind, seed if one_tree else seed + b) for b in range(B)]
    par = ints(parents[0] if one_tree else parents)
    out = attn.attn_decode_tree(q, kc, vc, par, cache_len=ints(lens) if lens is not None else None,
                                draft_len=ints(drafts) if drafts is not None else None, scale=scale)
    attn.attn_device_status()
    verify(q, kc, vc, parents, lens, drafts, out, scale, only, f"T {T} Skv {Skv} H {H}/{H_kv} D {D} {kind}")
    return q, kc, vc, parents, out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,H_kv", [(4, 4), (4, 2), (8, 1), (6, 2)])
@pytest.mark.parametrize("T,Skv", [(1, 1), (1, 700), (5, 64), (17, 300), (40, 1300), (63, 200), (64, 128), (128, 129),
                                   (100, 2000)])
def test_tree_bf16(gpu, T, Skv, H, H_kv, D):
    lens = [Skv, max(T, Skv // 2 + 3), min(Skv, T), T // 2, 0, min(Skv, T + 1)]
    drafts = [T, max(1, T // 2), T, T, T, T - 1]
    case(6, H, H_kv, T, Skv, D, lens, drafts, seed=T + Skv)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,H_kv", [(2, 2), (6, 2)])
@pytest.mark.parametrize("T,Skv", [(1, 1), (1, 300), (13, 64), (64, 500), (128, 300)])
def test_tree_fp32(gpu, T, Skv, H, H_kv, D):
    lens = [Skv, max(T, Skv // 2 + 3), min(Skv, T), T // 2, 0, min(Skv, T + 1)]
    drafts = [T, max(1, T // 2), T, T, T, T - 1]
    case(6, H, H_kv, T, Skv, D, lens, drafts, dtype=F32, seed=T + Skv)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["chain", "star", "binary"])
def test_shapes_of_trees(gpu, kind, dtype):
    for T in (2, 31, 33, 65, 127, 128):
        case(3, 4, 2, T, 400, 64, [400, 129, 256], None, kind, dtype, seed=T)
    case(3, 4, 2, 20, 400, 64, None, None, kind, dtype, seed=2, one_tree=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_draft_at_every_offset_of_a_tile(gpu, dtype):
    lens = [200 + i for i in range(66)]
    case(66, 2, 1, 70, 300, 64, lens, [70 - i % 3 for i in range(66)], dtype=dtype, seed=5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_split_at_every_offset_of_the_draft(gpu, dtype):
    """A long cache is split; the draft then lies in the last split, across two, or
    begins one, and a split may hold nothing."""
    Skv = 5000
    lens = [4096 + d for d in (-130, -64, -63, -1, 0, 1, 40, 63, 64, 65, 127, 128)] + [600, 90]
    case(len(lens), 2, 1, 96, Skv, 64, lens, [96, 50] * (len(lens) // 2), dtype=dtype, seed=6)


def test_long_cache(gpu):
    case(2, 8, 1, 40, 40000, 128, [40000, 31111], [40, 39], seed=7, only=(0, 5))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales(gpu, dtype):
    for scale in (0.0, 1.0):
        case(2, 4, 2, 20, 300, 64, [300, 100], [20, 9], dtype=dtype, scale=scale, seed=8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_chain_is_the_chunk_of_attn_fwd_chunked(gpu, dtype):
    B, H, H_kv, T, Skv, D = 4, 4, 2, 33, 500, 128
    q, kc, vc, parents, out = case(B, H, H_kv, T, Skv, D, [500, 100, 33, 12], None, "chain", dtype, seed=9)
    want = attn.attn_fwd_chunked(q.contiguous(), kc, vc, cache_len=ints([500, 100, 33, 12]))
    attn.attn_device_status()
    # each is within its own tolerance of the same definition
    err = (out.double() - want.double()).abs()
    assert err.max() <= (2 * 2.0 ** -6 if dtype == BF16 else 2e-4)
    assert torch.count_nonzero(out[3, :, :21]) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Skv", [300, 4000])
def test_masked_infinities_leave_no_trace(gpu, dtype, D, Skv):
    """Rows past the sequence's end and drafted tokens of other branches may hold
    infinities and NaN: rows that do not see them keep their bits."""
    B, H, H_kv, T = 3, 4, 2, 30
    lens, drafts = [Skv - 1, 150, 64], [30, 21, 30]
    q = wl.random_tensors((B, H, T, D), 10, dtype=dtype, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 11, dtype=dtype, count=2)
    parents = [tree(T, "random", 12 + b) for b in range(B)]
    call = lambda k, v: attn.attn_decode_tree(q, k, v, ints(parents), cache_len=ints(lens), draft_len=ints(drafts))  # noqa: E731
    clean = call(kc, vc)
    k2, v2 = kc.clone(), vc.clone()
    for b in range(B):
        k2[b, :, lens[b]:], v2[b, :, lens[b]:] = math.nan, math.inf
        past = lens[b] - drafts[b]
        k2[b, :, past + 9], v2[b, :, past + 9] = math.inf, math.nan
        v2[b, 0, past + 14, ::5] = -math.inf
    dirty = call(k2, v2)
    attn.attn_device_status()
    for b in range(B):
        see = sight(parents[b], lens[b], drafts[b])
        past = lens[b] - drafts[b]
        for h in range(H):
            hit = see[:, past + 9] | (see[:, past + 14] if h < 2 else False)
            n = drafts[b]
            assert torch.equal(dirty[b, h, :n][~hit], clean[b, h, :n][~hit]), (b, h)
            assert not torch.isfinite(dirty[b, h, :n][hit].float()).all(1).any()
            assert torch.count_nonzero(dirty[b, h, n:]) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_visible_infinities_are_kept(gpu, dtype):
    B, H, H_kv, T, Skv, D = 1, 2, 1, 25, 200, 64
    q = wl.random_tensors((B, H, T, D), 13, dtype=dtype, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 14, dtype=dtype, count=2)
    parents = [tree(T, "random", 15)]
    for row, col, x in ((199, 3, math.inf), (180, 3, -math.inf), (176, 40, math.inf), (20, 50, math.inf), (174, 60, -math.inf)):
        vc[0, 0, row, col] = x
    out = attn.attn_decode_tree(q, kc, vc, ints(parents))
    attn.attn_device_status()
    see = sight(parents[0], Skv, T).double()
    pos, neg = (see @ (vc[0, 0] == math.inf).double()) > 0, (see @ (vc[0, 0] == -math.inf).double()) > 0
    for h in range(H):
        got = out[0, h].float()
        assert torch.equal(torch.isnan(got), pos & neg)
        assert torch.equal(got == math.inf, pos & ~neg) and torch.equal(got == -math.inf, neg & ~pos)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_parents_and_lengths(gpu, dtype):
    """A parent that is not below its token counts as none; lengths are clamped."""
    B, H, H_kv, T, Skv, D = 4, 2, 1, 12, 100, 64
    q = wl.random_tensors((B, H, T, D), 16, dtype=dtype, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 17, dtype=dtype, count=2)
    parents = [[5, 1, 100, -7, 2000000000, 4, -2000000000, 7, 3, 0, 9, 11] for _ in range(B)]
    lens, drafts = [1000, -5, 7, 60], [12, 12, 99, -1]
    out = attn.attn_decode_tree(q, kc, vc, ints(parents), cache_len=ints(lens), draft_len=ints(drafts))
    attn.attn_device_status()
    verify(q, kc, vc, parents, lens, drafts, out)


def test_layouts_agree(gpu):
    B, H, H_kv, T, Skv, D = 2, 4, 2, 10, 300, 128
    q = wl.random_tensors((B, H, T, D), 18, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 19, count=2)
    par = ints(tree(T, "random", 20))
    a = attn.attn_decode_tree(q, kc, vc, par)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)   # token-major
    b = attn.attn_decode_tree(qt, kc, vc, par)
    assert b.stride() == qt.stride()
    fused = torch.zeros(B, T, H + 5, D, dtype=BF16, device="cuda")
    fused[:, :, 2:2 + H] = q.transpose(1, 2)
    out = torch.full((B, T, H + 1, D), 4.0, dtype=BF16, device="cuda")
    attn.attn_decode_tree(fused[:, :, 2:2 + H].transpose(1, 2), kc, vc, par, out=out[:, :, :H].transpose(1, 2))
    attn.attn_device_status()
    assert torch.equal(a, b) and torch.equal(out[:, :, :H].transpose(1, 2), a) and torch.all(out[:, :, H] == 4.0)


def test_offsets_past_32_bits(gpu):
    """A cache of 2.3e9 elements, the draft at its end."""
    B, H, H_kv, T, D = 2, 2, 1, 20, 128
    Skv = 9 << 20
    kc, vc = (torch.zeros((B, H_kv, Skv, D), dtype=BF16, device="cuda") for _ in range(2))
    q = wl.random_tensors((B, H, T, D), 21, count=1)[0]
    tk, tv = wl.random_tensors((B, H_kv, 4000, D), 22, count=2)
    kc[:, :, -4000:], vc[:, :, -4000:] = tk * 4, tv
    parents = [tree(T, "random", 23 + b) for b in range(B)]
    out = attn.attn_decode_tree(q, kc, vc, ints(parents), scale=1.0)
    attn.attn_device_status()
    verify(q, kc, vc, parents, None, None, out, scale=1.0, only=(0, 1))


def test_streams_graphs_and_two_calls_at_once(gpu):
    B, H, H_kv, T, Skv, D = 3, 8, 2, 20, 3000, 128
    sets = []
    for s in (30, 40):
        q = wl.random_tensors((B, H, T, D), s, count=1)[0]
        kc, vc = wl.random_tensors((B, H_kv, Skv, D), s + 1, count=2)
        par, cl, dl = ints([tree(T, "random", s + b) for b in range(B)]), ints([3000, 700, 2000]), ints([20, 5, 19])
        sets.append((q, kc, vc, par, cl, dl))
    want = [attn.attn_decode_tree(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(20):
        for x, s, w in zip(sets, streams, want):
            outs.append((attn.attn_decode_tree(*x, stream=s), w))
    torch.cuda.synchronize()
    attn.attn_device_status()
    for got, w in outs:
        assert torch.equal(got, w)
    graphs, bufs = [], [torch.empty_like(w) for w in want]
    for x, o in zip(sets, bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attn.attn_decode_tree(*x, out=o)
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(bufs, want):
        assert torch.equal(o, w)
    sets[0][4].copy_(ints([100, 20, 2999]))
    graphs[0].replay()
    torch.cuda.synchronize()
    attn.attn_device_status()
    assert torch.equal(bufs[0], attn.attn_decode_tree(*sets[0]))


def test_empty_calls_and_refusals(gpu):
    B, H, H_kv, T, Skv, D = 2, 4, 2, 6, 40, 64
    q = wl.random_tensors((B, H, T, D), 50, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 51, count=2)
    par = ints([tree(T, "chain", 0)] * B)
    assert attn.attn_decode_tree(q[:, :, :0], kc, vc, par[:, :0].contiguous()).shape == (B, H, 0, D)
    none = attn.attn_decode_tree(q, kc[:, :, :0].contiguous(), vc[:, :, :0].contiguous(), par)
    attn.attn_device_status()
    assert torch.count_nonzero(none) == 0
    for args in ((q, kc[:1], vc, par), (q, kc, vc, par[:, :5].contiguous()), (q, kc, vc, par.long()), (q, kc, vc, par.cpu()),
                 (q, kc.transpose(1, 2), vc, par), (q[0], kc, vc, par), (q.transpose(2, 3), kc, vc, par)):
        with pytest.raises(ValueError):
            attn.attn_decode_tree(*args)
    with pytest.raises(TypeError):
        attn.attn_decode_tree(q, kc.float(), vc.float(), par)
    with pytest.raises(ValueError):
        attn.attn_decode_tree(q, kc, vc, par, cache_len=ints([1, 2, 3]))
    big = torch.zeros(1, 2, 129, 64, dtype=BF16, device="cuda")
    with pytest.raises(attn.AttnError) as e:
        attn.attn_decode_tree(big, kc[:1], vc[:1], torch.zeros(129, dtype=torch.int32, device="cuda"))
    assert e.value.code == attn.ATTN_EUNSUPPORTED
    for kw in (dict(out=q), dict(scale=float("inf")), dict(out=torch.zeros(1, H, T, D, dtype=BF16, device="cuda").expand(B, H, T, D))):
        with pytest.raises(attn.AttnError) as e:
            attn.attn_decode_tree(q, kc, vc, par, **kw)
        assert e.value.code == attn.ATTN_EINVAL


# fp32: up to eight splits are a cluster (the sizes below give 1, 2, 4, 8 of them, some
# past a sequence's end), more leave their parts in the workspace
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Skv", [100, 129, 256, 257, 400, 513, 1024, 1025, 3000])
def test_fp32_splits(gpu, Skv, D):
    lens = [Skv, max(Skv // 2, 5), 5, 0, Skv - 1]
    T = 5
    case(len(lens), 6, 2, T, Skv, D, dtype=F32, lens=lens, drafts=[T, T, T, 0, 3], seed=Skv)


@pytest.mark.parametrize("G,T", [(1, 1), (1, 16), (1, 17), (2, 8), (4, 7), (1, 33)])
def test_fp32_rows_of_one_warp(gpu, G, T):
    case(2, 2 * G, 2, T, 300, 64, dtype=F32, lens=[300, 177], drafts=[T, max(T - 1, 1)], seed=T)


# more blocks than SMs: two blocks an SM, of half the workers; as clusters, alone, and
# with the workspace
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H_kv,T,Skv", [(90, 2, 3, 70), (40, 2, 9, 500), (24, 1, 40, 900), (12, 2, 5, 3000)])
def test_fp32_many_blocks(gpu, B, H_kv, T, Skv, D):
    lens = [max(0, Skv - 37 * b % Skv) for b in range(B)]
    case(B, 2 * H_kv, H_kv, T, Skv, D, lens, [min(T, n) for n in lens], dtype=F32, seed=B)


# a cache of one tile, several in one CTA or cluster, and one that many CTAs or splits share
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("B,Skv", [(1, 120), (3, 700), (1, 6000), (20, 1500)])
@pytest.mark.parametrize("draft_low", [False, True])
def test_a_seen_infinity_is_never_lost(gpu, dtype, B, Skv, T, draft_low):
    """Keys whose weights underflow (their scores lie some 1400 below the others) with
    infinite or NaN values: the element is infinite or NaN in every row that sees the
    key, wherever the cache is cut, and in no other."""
    H, H_kv, D = 4, 2, 64
    q = wl.random_tensors((B, H, T, D), 60, dtype=dtype, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 61, dtype=dtype, count=2)
    q[..., 0] = 8.0
    lens = [Skv - 3 * b for b in range(B)]
    parents = [tree(T, "random", 62 + b) for b in range(B)]
    for b in range(B):
        for row, col, x in ((3, 1, math.inf), (lens[b] // 2, 20, -math.inf), (lens[b] - T, 41, math.inf),
                            (lens[b] - T + 2, 50, math.nan), (lens[b] - 1, 7, -math.inf)):
            kc[b, :, row, 0] = -180.0 * math.sqrt(D)
            vc[b, :, row, col] = x
        if draft_low:  # every drafted key: a part of the draft alone has a maximum far below the others'
            kc[b, :, lens[b] - T:lens[b], 0] = -180.0 * math.sqrt(D)
    out = attn.attn_decode_tree(q, kc, vc, ints(parents), cache_len=ints(lens))
    attn.attn_device_status()
    for b in range(B):
        see = sight(parents[b], lens[b], T)
        for h in range(H):
            hit = (see.double() @ (~torch.isfinite(vc[b, h // 2, :lens[b]])).double()) > 0
            assert torch.equal(~torch.isfinite(out[b, h]), hit), (b, h)
            o, _, A, size = ref.attend(q[b, h], kc[b, h // 2, :lens[b]], vc[b, h // 2, :lens[b]], see, D ** -0.5)
            tol, _ = ref.bounds(dtype, D, lens[b], D ** -0.5, size, o, A)
            zero = torch.zeros_like(o)
            ref.check(torch.where(hit, zero, out[b, h].double()), torch.where(hit, zero, o), tol)



@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,T", [(64, 30), (128, 70)])
@pytest.mark.parametrize("Skv", [200, 4000])
def test_huge_scores_stay_in_their_rows(gpu, dtype, D, T, Skv):
    """Scores of huge or infinite magnitude of a drafted key or query: the rows that
    have no part in them keep their bits."""
    B, H, H_kv = 3, 4, 2
    lens, drafts = [Skv - 1, 150, 64], [T, 21, min(T, 30)]
    q = wl.random_tensors((B, H, T, D), 63, dtype=dtype, count=1)[0]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 64, dtype=dtype, count=2)
    parents = [tree(T, "random", 65 + b) for b in range(B)]
    call = lambda q, k: attn.attn_decode_tree(q, k, vc, ints(parents), cache_len=ints(lens), draft_len=ints(drafts))  # noqa: E731
    clean = call(q, kc)
    for x in (1e9, -1e9, math.inf, -math.inf):
        k2, q2 = kc.clone(), q.clone()
        for b in range(B):
            k2[b, :, lens[b] - drafts[b] + 9, 3] = x
            q2[b, :, 13, 3] = x
        by_key, by_query = call(q, k2), call(q2, kc)
        attn.attn_device_status()
        for b in range(B):
            n = drafts[b]
            hidden = ~sight(parents[b], lens[b], n)[:, lens[b] - n + 9]
            assert torch.equal(by_key[b, :, :n][:, hidden], clean[b, :, :n][:, hidden]), (x, b)
            other = torch.arange(T, device="cuda") != 13
            assert torch.equal(by_query[b][:, other], clean[b][:, other]), (x, b)


# one tile, several tiles in a CTA, many CTAs or splits a unit; one and two row tiles
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,T", [(64, 30), (128, 70)])
@pytest.mark.parametrize("B,Skv", [(2, 120), (40, 500), (1, 6000)])
def test_distinct_scores_of_huge_magnitude(gpu, dtype, D, T, B, Skv):
    """Scores of 2^27 to 2^92 of both signs, growing over the tiles, beside rows of zeros."""
    H, H_kv = 4, 2
    vc = wl.random_tensors((B, H_kv, Skv, D), 66, dtype=dtype, count=1)[0]
    q = torch.zeros(B, H, T, D, dtype=dtype, device="cuda")
    kc = torch.zeros(B, H_kv, Skv, D, dtype=dtype, device="cuda")
    for b in range(B):
        for h in range(H):
            q[b, h] = ref.huge_inputs(T, Skv, D, dtype, 67 + 8 * b + h)[0]
        for g in range(H_kv):
            kc[b, g] = ref.huge_inputs(T, Skv, D, dtype, 167 + 8 * b + g)[1]
    lens = [Skv - 3 * b for b in range(B)]
    parents = [tree(T, "random", 68 + b) for b in range(B)]
    out = attn.attn_decode_tree(q, kc, vc, ints(parents), cache_len=ints(lens), scale=1.0)
    attn.attn_device_status()
    for b in range(B):
        see = sight(parents[b], lens[b], T)
        for h in range(H):
            ref.check_huge(out[b, h], None, q[b, h], kc[b, h // 2, :lens[b]], vc[b, h // 2, :lens[b]], see, dtype, f"{b} {h}")
