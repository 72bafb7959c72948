"""GPU tests of attn_fwd_paged against the definition in 64 bits; the tolerances are
derived in serving_ref.py.  Whatever no token may see is NaN in the pools: rows past a
sequence's end, pages of nobody, and what the tables hold behind their pages is no page."""
from __future__ import annotations

import math
import random

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Paged:
    """A pool with sequences of (keys, new tokens) in pages drawn at random."""

    def __init__(self, seqs, H, H_kv, D, P, dtype=BF16, seed=1, layout="heads", junk=math.nan, front=0, back=0, even=None):
        r = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.H_kv, self.D, self.P, self.dtype = seqs, H, H_kv, D, P, dtype
        counts = [-(-L // P) for L, _ in seqs]
        self.n_pages = n_pages = sum(counts) + 3
        self.M = max(counts, default=0) + 2
        shape = {"heads": (n_pages, H_kv, P, D), "rows": (n_pages, P, H_kv, D), "halves": (n_pages, 2, H_kv, P, D),
                 "apart": (n_pages, H_kv * P * D + 64), "by head": (H_kv, n_pages, P, D)}[layout]
        pools = [torch.full(shape, junk, dtype=dtype, device="cuda") for _ in range(1 if layout == "halves" else 2)]
        if layout == "heads":
            self.kp, self.vp = pools
        elif layout == "apart":  # the heads of all pages are not evenly spaced
            self.kp, self.vp = (x[:, :H_kv * P * D].view(n_pages, H_kv, P, D) for x in pools)
        elif layout == "by head":
            self.kp, self.vp = (x.transpose(0, 1) for x in pools)
        elif layout == "rows":
            self.kp, self.vp = (x.transpose(1, 2) for x in pools)
        else:
            self.kp, self.vp = pools[0][:, 0], pools[0][:, 1]
        ids = list(range(n_pages))
        r.shuffle(ids)
        table = [[r.choice((-1, n_pages, 2 ** 31 - 1, -2 ** 31)) for _ in range(self.M)] for _ in seqs]
        self.k, self.v = [], []
        for b, (L, _) in enumerate(seqs):
            k, v = (torch.randn(L, H_kv, D, generator=g).to(dtype).cuda() for _ in range(2))
            self.k.append(k), self.v.append(v)
            for p in range(counts[b]):
                page = table[b][p] = ids.pop()
                rows = slice(p * P, min(L, (p + 1) * P))
                n = rows.stop - rows.start
                self.kp[page, :, :n], self.vp[page, :, :n] = k[rows].transpose(0, 1), v[rows].transpose(0, 1)
        self.table, self.lens = ints(table), ints([L for L, _ in seqs])
        self.ends = [front]
        for _, n in seqs:
            self.ends.append(self.ends[-1] + n)
        self.T = self.ends[-1] + back
        self.cu = None if even else ints(self.ends)
        self.q = torch.randn(self.T, H, D, generator=g).to(dtype).cuda()

    def call(self, **kw):
        return attn.attn_fwd_paged(self.q, self.kp, self.vp, self.table, self.lens, cu_seqlens=self.cu, **kw)

    def check(self, out, lse=None, scale=None, heads=None, what=""):
        scale = self.D ** -0.5 if scale is None else scale
        G = self.H // self.H_kv
        for b, (L, n) in enumerate(self.seqs):
            if n == 0:
                continue
            rows = slice(self.ends[b], self.ends[b + 1])
            see = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda")[:, None]
            some = see.any(1)
            empty = torch.nonzero(~some)[:, 0] + self.ends[b]
            assert torch.count_nonzero(out[empty]) == 0, f"{what}: a row without a key"
            if lse is not None:
                assert bool((lse[empty] == -math.inf).all())
            if not bool(some.any()):
                continue
            for h in range(self.H) if heads is None else heads:
                o, l, A, size = ref.attend(self.q[rows, h][some], self.k[b][:, h // G], self.v[b][:, h // G], see[some], scale)
                tol, ltol = ref.bounds(self.dtype, self.D, L, scale, size, o, A)
                ref.check(out[rows, h][some], o, tol, f"{what} sequence {b} (L {L}, n {n}) head {h}")
                if lse is not None:
                    err = (lse[rows, h][some].double() - l).abs()
                    assert torch.all(err <= ltol + l.abs() * 2.0 ** -21), f"{what} lse of sequence {b}: {err.max():.3e}"


SEQS = [(1, 1), (130, 1), (77, 77), (300, 45), (0, 0), (513, 130), (128, 128), (5, 0), (1000, 3), (257, 1), (256, 64)]


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("H,H_kv", [(4, 4), (8, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("P", [8, 16, 64, 256, 24])
def test_chunks_and_tokens(gpu, P, H, H_kv, dtype, D):
    x = Paged(SEQS, H, H_kv, D, P, dtype, seed=P + H)
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse, what=f"P {P} H {H}/{H_kv}")


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("H,H_kv", [(4, 4), (32, 8), (12, 4), (16, 1)])
@pytest.mark.parametrize("lens", [[1], [1500], [128, 1, 129, 127, 0, 8192], list(range(1, 400, 6))])
def test_single_tokens(gpu, lens, H, H_kv, dtype, D):
    for n in (1, 3):
        x = Paged([(L, n) for L in lens], H, H_kv, D, 16, dtype, seed=len(lens) + n, even=True)
        out, lse = x.call(return_lse=True)
        attn.attn_device_status()
        x.check(out, lse, heads=(0, H - 1), what=f"{n} a sequence")


@pytest.mark.parametrize("H_kv", [1, 2, 8])
@pytest.mark.parametrize("B", [1, 2, 3, 4, 9, 16, 19, 37, 75])
@pytest.mark.parametrize("longest", [60, 700, 2100])
def test_a_few_sequences(gpu, longest, B, H_kv):
    """One to a few hundred units: clusters of eight, four, two and one CTAs, and none."""
    lens = [longest] + [(37 * b * b) % (longest + 1) for b in range(1, B)]
    for n, D in ((1, 128), (2, 64)):
        x = Paged([(L, n) for L in lens], 2 * H_kv, H_kv, D, 16, BF16, seed=B + longest, even=True)
        out, lse = x.call(return_lse=True)
        attn.attn_device_status()
        x.check(out, lse, heads=(0, 2 * H_kv - 1), what=f"{B} sequences of {n}")
        assert torch.equal(x.call(), out)


@pytest.mark.parametrize("H,H_kv", [(33, 1), (128, 1), (130, 1), (200, 1), (260, 2), (600, 2)])
def test_large_groups(gpu, H, H_kv):
    for dtype in (BF16, F32):
        x = Paged([(140, 5), (1, 1), (300, 1)], H, H_kv, 64, 32, dtype, seed=H)
        out, lse = x.call(return_lse=True)
        attn.attn_device_status()
        x.check(out, lse, heads=(0, 1, 127 % H, 128 % H, 129 % H, H - 1), what=f"H {H}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_offset_of_the_last_key(gpu, dtype):
    """Sequence ends and diagonals at every place of a tile and of a page."""
    seqs = [(180 + i, 1 + i % 70) for i in range(132)]
    x = Paged(seqs, 2, 1, 64, 16, dtype, seed=3)
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse)


@pytest.mark.parametrize("dtype,L,n", [(BF16, 20011, 1), (BF16, 9000, 1300), (F32, 9001, 1), (F32, 3001, 90)])
def test_long_sequences_are_split(gpu, dtype, L, n):
    x = Paged([(L, n)], 4, 1, 128 if dtype == BF16 else 64, 64, dtype, seed=L)
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse, heads=(0, 3))
    again, lse2 = x.call(return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["rows", "halves", "apart", "by head"])
@pytest.mark.parametrize("P,D", [(16, 64), (16, 128), (256, 128)])
def test_strides_of_pages(gpu, P, D, layout, dtype):
    x = Paged(SEQS, 8, 4, D, P, dtype, seed=9, layout=layout)
    y = Paged(SEQS, 8, 4, D, P, dtype, seed=9)
    a, la = x.call(return_lse=True)
    b, lb = y.call(return_lse=True)
    attn.attn_device_status()
    x.check(a, la)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows_tables_and_given_outputs(gpu, dtype):
    x = Paged(SEQS, 4, 2, 64, 16, dtype, seed=11)
    want, lse = x.call(return_lse=True)
    wide = torch.zeros(x.T, 10, 64, dtype=dtype, device="cuda")
    wide[:, 2:6] = x.q
    table = torch.full((len(SEQS), x.M + 5), 7, dtype=torch.int32, device="cuda")
    table[:, :x.M] = x.table
    out = torch.full((x.T, 9, 64), 3.0, dtype=dtype, device="cuda")
    lse2 = torch.empty_like(lse)
    x.q, x.table = wide[:, 2:6], table[:, :x.M]
    got = x.call(out=out[:, 5:9], lse=lse2)
    attn.attn_device_status()
    assert got[0].data_ptr() == out[:, 5:9].data_ptr() and got[1] is lse2
    assert torch.equal(out[:, 5:9], want) and torch.equal(lse2, lse) and bool((out[:, :5] == 3).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_outside_every_sequence_stay(gpu, dtype):
    x = Paged([(40, 3), (0, 0), (200, 130)], 4, 2, 64, 16, dtype, seed=4, front=37, back=50)
    out, lse = torch.full_like(x.q, 5.0), torch.full((x.T, 4), 5.0, device="cuda")
    x.call(out=out, lse=lse)
    attn.attn_device_status()
    x.check(out, lse)
    for t in (out, lse):
        assert bool((t[:37] == 5).all()) and bool((t[-50:] == 5).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tokens_in_front_of_the_first_key(gpu, dtype):
    """Fewer keys than new tokens: the first tokens see nothing."""
    x = Paged([(3, 10), (0, 5), (1, 200), (130, 131), (0, 1)], 4, 2, 64, 16, dtype, seed=6)
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_pages_at_all(gpu, dtype):
    q = torch.randn(3, 4, 64, device="cuda").to(dtype)
    pages = torch.empty(0, 2, 16, 64, dtype=dtype, device="cuda")
    out, lse = attn.attn_fwd_paged(q, pages, pages, torch.empty(3, 0, dtype=torch.int32, device="cuda"), return_lse=True)
    attn.attn_device_status()
    assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())
    none = attn.attn_fwd_paged(q[:0], pages, pages, torch.empty(0, 4, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_are_clamped_and_default_to_the_table(gpu, dtype):
    P = 16
    x = Paged([(64, 2), (64, 2)], 4, 2, 64, P, dtype, seed=8, even=True)
    x.table = x.table[:, :4].contiguous()  # full rows
    want = x.call()
    assert torch.equal(attn.attn_fwd_paged(x.q, x.kp, x.vp, x.table), want)
    x.lens = ints([1000, 64])
    assert torch.equal(x.call(), want)
    x.lens = ints([64, -7])
    got = x.call()
    attn.attn_device_status()
    assert torch.equal(got[:2], want[:2]) and torch.count_nonzero(got[2:]) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_entries_that_are_no_pages_read_as_zeros(gpu, dtype):
    x = Paged([(200, 40), (100, 1)], 4, 2, 64, 16, dtype, seed=12)
    for b, p, bad in ((0, 3, -1), (0, 12, x.n_pages), (1, 0, 2 ** 31 - 1), (1, 6, -2 ** 31)):
        x.table[b, p] = bad
        for t in (x.k[b], x.v[b]):
            t[16 * p:16 * (p + 1)] = 0
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_pages(gpu, dtype):
    """Two sequences over the same first pages, each as if they were its own."""
    x = Paged([(70, 5), (70, 1), (64, 64)], 4, 2, 64, 16, dtype, seed=13)
    x.table[1, :4] = x.table[0, :4]
    x.k[1][:64], x.v[1][:64] = x.k[0][:64], x.v[0][:64]
    x.table[2, :4] = x.table[0, :4]
    x.k[2], x.v[2] = x.k[0][:64], x.v[0][:64]
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_nonfinite_values_go_to_the_rows_that_see_them(gpu, value, dtype):
    x = Paged([(300, 150), (129, 1)], 4, 2, 64, 16, dtype, seed=14)
    clean = x.call()
    for j in (20, 200, 255, 299):
        page = int(x.table[0, j // 16])
        x.vp[page, 1, j % 16, 7] = value
        x.v[0][j, 1, 7] = value
    out = x.call()
    attn.attn_device_status()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:150, 2:, 7] = True  # key 20 is seen by all rows of the second cached head
    assert torch.equal(out[~hit], clean[~hit])
    got = out[hit].float()
    assert bool(got.isnan().all()) if math.isnan(value) else bool((got.isnan() | (got == value)).all())
    x.vp[int(x.table[0, 1]), 1, 4, 7] = 0.25  # key 20
    out = x.call()
    first = 200 - 150  # the first token that sees key 200
    assert bool(out[:first, 2:, 7].isfinite().all()) and not bool(out[first:150, 2:, 7].isfinite().any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,H_kv,B", [(4, 2, 1), (4, 2, 40), (24, 1, 1), (24, 1, 40), (96, 2, 1), (96, 2, 30)])
def test_nonfinite_values_and_single_tokens(gpu, H, H_kv, B, dtype):
    """Few and many sequences, few rows a tile and many: the values reach every head of their group,
    and none of those past the end, of the other group or of a neighbour."""
    lens = [700, 129, 257, 64, 1, 300]
    x = Paged([(lens[b % 6], 1) for b in range(B)], H, H_kv, 64, 16, dtype, seed=14, even=True)
    clean = x.call()
    G = H // H_kv
    for b, j, value in ((0, 699, math.inf), (0, 3, -math.inf), (B - 1, 0, math.nan)):
        x.vp[int(x.table[b, j // 16]), H_kv - 1, j % 16, 9 + b % 2] = value
    out = x.call()
    attn.attn_device_status()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, H - G:, 9] = True
    hit[B - 1, H - G:, 9 + (B - 1) % 2] = True
    assert torch.equal(out[~hit], clean[~hit]) and not bool(out[hit].isfinite().any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,G", [(1, 4), (1, 40), (50, 4)])
def test_huge_scores_of_single_tokens(gpu, B, G, dtype):
    L, D = 400, 64
    x = Paged([(L, 1)] * B, G, 1, D, 16, dtype, seed=15, even=True)
    q, k = ref.huge_inputs(B * G, L, D, dtype, 3)
    for b in range(B):
        pages = x.table[b, :L // 16].long()
        x.kp[pages, 0] = k.view(-1, 16, D)
        x.vp[pages, 0] = x.v[b][:, 0].view(-1, 16, D)
    x.q = q.view(B, G, D)
    out, lse = x.call(scale=1.0, return_lse=True)
    attn.attn_device_status()
    see = torch.ones(G, L, dtype=torch.bool, device="cuda")
    for b in range(B):
        ref.check_huge(out[b], lse[b], x.q[b], k, x.v[b][:, 0], see, dtype)


@pytest.mark.parametrize("H,H_kv", [(8, 2), (32, 1), (33, 1), (20, 2), (64, 1)])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 33])
def test_a_few_rows(gpu, n, H, H_kv):
    """Numbers of rows around those that share a tile's columns among four warps, one sequence and many, chunks beside them."""
    for seqs in ([(1500, n)], [(n, n)], [(n - 1, n)], [(200 + 7 * i, n) for i in range(20)], [(300, n), (900, 100), (17, 1), (260, n)]):
        x = Paged(seqs, H, H_kv, 128 if H < 33 else 64, 16, seed=n + H)
        out, lse = x.call(return_lse=True)
        attn.attn_device_status()
        x.check(out, lse, heads=(0, H // H_kv - 1, H - 1), what=f"n {n} H {H}/{H_kv} {seqs[:2]}")


def _into_pages(x, b, k, v):
    for j in range(k.shape[0]):
        page = int(x.table[b, j // x.P])
        x.kp[page, 0, j % x.P], x.vp[page, 0, j % x.P] = k[j], v[j]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_huge_scores(gpu, dtype):
    L, n, D = 400, 40, 64
    x = Paged([(L, n)], 1, 1, D, 16, dtype, seed=15)
    q, k = ref.huge_inputs(n, L, D, dtype, 3)
    _into_pages(x, 0, k, x.v[0][:, 0])
    x.q = q[:, None].contiguous()
    out, lse = x.call(scale=1.0, return_lse=True)
    attn.attn_device_status()
    see = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda")[:, None]
    ref.check_huge(out[:, 0], lse[:, 0], q, k, x.v[0][:, 0], see, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [math.inf, math.nan, 1e30])
@pytest.mark.parametrize("seqs", [[(300, 20), (500, 40), (700, 1), (64, 64), (1000, 3)], [(900, 1), (900, 1), (100, 1), (20, 1), (5, 1)]])
def test_tokens_of_other_sequences_leave_no_trace(gpu, seqs, value, dtype):
    """A tile's rows behind its sequence's last token are other sequences' tokens, or nothing."""
    x = Paged(seqs, 8, 2, 128, 16, dtype, seed=11)
    out, lse = x.call(return_lse=True)
    for b in range(len(seqs)):
        rows = slice(x.ends[b], x.ends[b + 1])
        kept, x.q = x.q, x.q.clone()
        x.q[rows] = value
        got, got_lse = x.call(return_lse=True)
        x.q = kept
        others = torch.ones(x.T, dtype=torch.bool, device="cuda")
        others[rows] = False
        assert torch.equal(got[others], out[others]) and torch.equal(got_lse[others], lse[others])
    attn.attn_device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_of_zero_is_the_mean(gpu, dtype):
    x = Paged([(300, 45), (1, 1), (131, 1)], 4, 2, 64, 16, dtype, seed=16)
    out, lse = x.call(scale=0.0, return_lse=True)
    attn.attn_device_status()
    x.check(out, lse, scale=0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_with_new_tables_and_lengths(gpu, dtype):
    """A captured call reads tables, lengths and offsets when it is replayed."""
    x = Paged([(400, 30), (300, 1), (200, 1), (64, 32)], 8, 2, 64, 16, dtype, seed=17)
    x.call(return_lse=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = x.call(return_lse=True)
    for seqs in ([(400, 30), (300, 1), (200, 1), (64, 32)], [(31, 1), (1, 1), (350, 61), (0, 1)], [(380, 64), (0, 0), (0, 0), (0, 0)]):
        y = Paged(seqs, 8, 2, 64, 16, dtype, seed=18)
        x.q.copy_(y.q), x.lens.copy_(y.lens), x.cu.copy_(y.cu), x.table[:, :y.M].copy_(y.table)
        x.kp[:y.n_pages].copy_(y.kp), x.vp[:y.n_pages].copy_(y.vp)
        g.replay()
        torch.cuda.synchronize()
        attn.attn_device_status()
        y.check(out, lse)


def test_two_streams_at_once(gpu):
    xs = [Paged([(900 + 300 * i, 200), (500, 1)], 8, 2, 128, 32, seed=20 + i) for i in range(3)]
    want = [x.call() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(20):
        for x, s, g in zip(xs, streams, got):
            with torch.cuda.stream(s):
                g.append(x.call())
    torch.cuda.synchronize()
    attn.attn_device_status()
    for w, g in zip(want, got):
        assert all(torch.equal(w, y) for y in g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = xs[0].call(stream=side)
    side.synchronize()
    assert torch.equal(other, want[0])


def test_many_sequences(gpu):
    """More sequences than a warp has lanes, most of them empty or one token."""
    r = random.Random(2)
    seqs = [(L, n if L else 0) for L, n in ((r.randint(0, 200), r.choice((0, 1, 1, 1, 17))) for _ in range(333))]
    for dtype in (BF16, F32):
        x = Paged(seqs, 4, 2, 64, 16, dtype, seed=30)
        out, lse = x.call(return_lse=True)
        attn.attn_device_status()
        x.check(out, lse, heads=(0, 3))


def test_pools_past_32_bits(gpu):
    """Pages whose elements lie past 2^31 and whose bytes past 2^32."""
    P, H_kv, D = 256, 8, 128
    n_pages = (1 << 31) // (P * H_kv * D) + 20
    for dtype in (BF16, F32):
        kp, vp = (torch.zeros(n_pages, H_kv, P, D, dtype=dtype, device="cuda") for _ in range(2))
        x = Paged([(700, 3), (256, 1)], 16, H_kv, D, P, dtype, seed=31)
        far = [n_pages - 1 - i for i in range(x.n_pages)]
        kp[torch.tensor(far)], vp[torch.tensor(far)] = x.kp, x.vp
        x.table = torch.where((x.table >= 0) & (x.table < x.n_pages), n_pages - 1 - x.table, x.table)
        x.kp, x.vp = kp, vp
        out = x.call()
        attn.attn_device_status()
        x.check(out, heads=(0, 7, 15))
        del kp, vp, x
