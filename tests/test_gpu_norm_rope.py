"""GPU tests of attn_norm_rope and attn_rope_append_paged against the definition in 64 bits.

Tolerance.  The sum of a row's squares is a chain of at most 16 FMAs and 5 additions a
lane, each off by 2^-24: 21 * 2^-24 of the sum, half of that in its root; rsqrtf is good to 2
ulp (2^-22), the FMA with eps and the two products with the row's factor and the weight add
2^-25 + 2 * 2^-24: a normed element is off by 1.1e-6 of itself.  The turn adds 5e-7 mscale
(|a| + |b|) (test_gpu_rope.py).  Together 1.6e-6 mscale (|a| + |b|) of the normed pair, and
one rounding to the output type (2^-8 of the value for bf16)."""
from __future__ import annotations

import math
import random

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from test_gpu_rope import ints, rows, turned

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def normed(x, w, eps):
    x = x.detach().cpu().double()
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.cpu().double()


def check(got, x, w, eps, pos, f, interleaved=False, mscale=1.0, what=""):
    y = normed(x, w, eps)
    want, size = turned(y, pos, f, interleaved, False, mscale)
    tol = torch.where(size > 0, 1.6e-6 * abs(mscale) * size, 1.1e-6 * y.abs() if w is not None else torch.zeros_like(y))
    if got.dtype == BF16:
        tol = tol + (want.abs() + tol) * (torch.finfo(BF16).eps / 2)
    err = (got.cpu().double() - want).abs()
    assert torch.all(err <= tol), f"{what}: worst excess {(err - tol).max():.3e}"


def weights(D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 64), (128, 36), (128, 2), (128, 0), (64, 64), (64, 48), (64, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(gpu, dtype, D, rd, interleaved):
    T, H, H_kv = 37, 6, 2
    q, k = rows(T, H, D, 1, dtype), rows(T, H_kv, D, 2, dtype)
    k *= 100.0
    pos = torch.randint(-50, 1 << 21, (T,), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    f = attn.attn_rope_frequencies(rd)
    wq, wk = weights(D, dtype, 4)
    qo, ko = attn.attn_norm_rope(q, k, pos, f, wq, wk, eps=1e-5, interleaved=interleaved, mscale=1.25)
    check(qo, q, wq, 1e-5, pos, f, interleaved, 1.25, "q")
    check(ko, k, wk, 1e-5, pos, f, interleaved, 1.25, "k")


@pytest.mark.parametrize("T", [1, 2, 303, 5000, 10001])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (32, 8), (5, 0), (130, 1)])
def test_sizes(gpu, T, H, H_kv):
    q = rows(T, H, 128, 4, BF16)
    k = rows(T, H_kv, 128, 5, BF16) if H_kv else None
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    f = attn.attn_rope_frequencies(128, theta=500000.0)
    wq, wk = weights(128, BF16, 6)
    out = attn.attn_norm_rope(q, k, pos, f, wq, wk if H_kv else None)
    for x, w, got in zip((q, k), (wq, wk), out if H_kv else (out,)):
        check(got, x, w, 1e-6, pos, f)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rd,interleaved", [(64, False), (36, False), (36, True)])
def test_in_place_on_slices_and_without_a_weight(gpu, dtype, rd, interleaved):
    """Only q is normed; k is turned as attn_rope turns it; both in place."""
    T, H, H_kv, D = 50, 4, 2, 64
    qkv = rows(T, H + 2 * H_kv, D, 7, dtype)
    keep = qkv.clone()
    q, k = qkv[:, :H], qkv[:, H:H + H_kv]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f, wq = attn.attn_rope_frequencies(rd), weights(D, dtype, 8)[0]
    got = attn.attn_norm_rope(q, k, pos, f, wq, None, q_out=q, k_out=k, interleaved=interleaved)
    assert got[0] is q and got[1] is k
    check(q, keep[:, :H], wq, 1e-6, pos, f, interleaved)
    check(k, keep[:, H:H + H_kv], None, 1e-6, pos, f, interleaved)
    assert torch.equal(qkv[:, H + H_kv:], keep[:, H + H_kv:])
    assert torch.equal(k[..., rd:], keep[:, H:H + H_kv, rd:])


def test_element_aligned_rows(gpu):
    """Pointers and strides of single elements."""
    T, H, D = 21, 3, 128
    for dtype in (BF16, F32):
        buf = rows(T, H * (D + 3) + 5, 1, 9, dtype).view(T, -1)
        q = buf[:, 1:1 + H * (D + 3)].view(T, H, D + 3)[..., :D]
        w = torch.ones(D + 1, dtype=dtype, device="cuda")[1:]
        w[3] = 2.0
        pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), attn.attn_rope_frequencies(D)
        check(attn.attn_norm_rope(q, None, pos, f, w), q, w, 1e-6, pos, f)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_without_size(gpu, dtype):
    """Zeros stay zeros (with eps), tiny rows are lifted as eps allows, an infinity hurts its own row only."""
    q = rows(8, 2, 64, 10, dtype)
    q[1] = 0
    q[2] = q[2] * 1e-6
    q[3, 0, 5] = math.inf
    w = weights(64, dtype, 11)[0]
    pos, f = torch.arange(8, dtype=torch.int32, device="cuda"), attn.attn_rope_frequencies(32)
    got = attn.attn_norm_rope(q, None, pos, f, w, eps=1e-6)
    assert torch.count_nonzero(got[1]) == 0
    assert bool(got[3, 0].isnan().any()) and bool(got[3, 1].isfinite().all())
    keep = torch.ones(8, 2, dtype=torch.bool, device="cuda")
    keep[3, 0] = False
    some = keep.all(1).nonzero()[:, 0]
    check(got[some], q[some], w, 1e-6, pos[some], f)
    assert bool(attn.attn_norm_rope(q, None, pos, f, w, eps=0.0)[1].isnan().all())


def test_an_infinite_pair_past_the_turned_ones_stays(gpu):
    """In the unit where the turned pairs end, the others are left alone."""
    for dtype in (BF16, F32):
        q = rows(3, 2, 64, 12, dtype)
        q[1, 1, 36] = math.inf  # the first element past rotary_dim
        pos, f = ints([3, 4, 5]), attn.attn_rope_frequencies(36)
        got = attn.attn_norm_rope(q, None, pos, f, interleaved=True)
        assert torch.equal(got[..., 36:], q[..., 36:])
        assert bool(got[..., :36].isfinite().all())


# ------------------------------------------------------------ into pages

class Append:
    def __init__(self, seqs, H, H_kv, D, P, dtype, seed, layout="heads", junk=7.0, front=0, back=0, even=False):
        r = random.Random(seed)
        self.seqs, self.P, self.H, self.H_kv = seqs, P, H, H_kv
        counts = [-(-max(L, 0) // P) for L, _ in seqs]
        self.n_pages = sum(counts) + 2
        shape = (self.n_pages, P, H_kv, D) if layout == "rows" else (self.n_pages, 2, H_kv, P, D) if layout == "halves" else (self.n_pages, H_kv, P, D)
        pools = [torch.full(shape, junk, dtype=dtype, device="cuda") for _ in range(1 if layout == "halves" else 2)]
        self.kp, self.vp = (pools[0][:, 0], pools[0][:, 1]) if layout == "halves" else pools if layout == "heads" else [p.transpose(1, 2) for p in pools]
        ids = list(range(self.n_pages))
        r.shuffle(ids)
        self.M = max(counts) + 2
        self.table_l = [[ids.pop() if p < counts[b] else r.choice((-1, self.n_pages, 2 ** 31 - 1)) for p in range(self.M)] for b in range(len(seqs))]
        self.table, self.lens = ints(self.table_l), ints([L for L, _ in seqs])
        self.ends = [front]
        for _, n in seqs:
            self.ends.append(self.ends[-1] + n)
        T = self.ends[-1] + back
        self.cu = None if even else ints(self.ends)
        qkv = rows(T, H + 2 * H_kv, D, seed, dtype)
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]

    def positions(self):
        pos = torch.zeros(self.q.shape[0], dtype=torch.int32)
        for b, (L, n) in enumerate(self.seqs):
            pos[self.ends[b]:self.ends[b + 1]] = torch.arange(L - n, L)
        return pos.cuda()

    def call(self, f, **kw):
        return attn.attn_rope_append_paged(self.q, self.k, self.v, self.kp, self.vp, self.table, f, self.lens,
                                           cu_seqlens=self.cu, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rd,interleaved", [(128, 128, False), (64, 64, True), (64, 36, False), (128, 20, True)])
@pytest.mark.parametrize("P,layout", [(16, "heads"), (8, "rows"), (64, "halves"), (1, "heads"), (37, "rows")])
@pytest.mark.parametrize("norm", [True, False])
def test_append(gpu, dtype, D, rd, interleaved, P, layout, norm):
    x = Append([(70, 70), (0, 0), (131, 1), (16, 3), (3, 8), (200, 90), (0, 2)], 6, 2, D, P, dtype, seed=P, layout=layout, front=3,
               back=4)
    f = attn.attn_rope_frequencies(rd)
    wq, wk = weights(D, dtype, 5) if norm else (None, None)
    before = x.kp.clone(), x.vp.clone()
    k_out = torch.full((x.k.shape[0], 2, D), 5.0, dtype=dtype, device="cuda")
    q_out = torch.full((x.k.shape[0], 6, D), 5.0, dtype=dtype, device="cuda")
    got = x.call(f, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved, k_out=k_out, q_out=q_out)
    attn.attn_device_status()
    assert got[0] is q_out and got[1] is k_out
    pos, mine = x.positions(), slice(x.ends[0], x.ends[-1])
    check(q_out[mine], x.q[mine], wq, 1e-5, pos[mine], f, interleaved, what="q")
    check(k_out[mine], x.k[mine], wk, 1e-5, pos[mine], f, interleaved, what="k")
    for t in (q_out, k_out):
        assert bool((t[:3] == 5).all()) and bool((t[-4:] == 5).all())
    want = before
    for b, (L, n) in enumerate(x.seqs):
        for i in range(n):
            j = L - n + i
            if j >= 0:
                page = x.table_l[b][j // P]
                want[0][page, :, j % P] = k_out[x.ends[b] + i]
                want[1][page, :, j % P] = x.v[x.ends[b] + i]
    assert torch.equal(x.kp, want[0]) and torch.equal(x.vp, want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_and_contiguous_cache_as_pages(gpu, dtype):
    """One token each, positions given; a contiguous cache is one page a sequence: as attn_rope_append."""
    B, H, H_kv, D, Skv = 5, 4, 2, 64, 50
    qkv = rows(B, H + 2 * H_kv, D, 3, dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    lens, pos, f = ints([1, 50, 7, 0, 33]), ints([9, 8, 100, 3, 5]), attn.attn_rope_frequencies(D)
    a = [torch.zeros(B, H_kv, Skv, D, dtype=dtype, device="cuda") for _ in range(2)]
    b = [torch.zeros(B, H_kv, Skv, D, dtype=dtype, device="cuda") for _ in range(2)]
    qa = attn.attn_rope_append(q, k, v, *a, f, cache_len=lens, positions=pos)
    qb = attn.attn_rope_append_paged(q, k, v, *b, ints([[i] for i in range(B)]), f, lens, positions=pos)
    assert torch.equal(qa, qb) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_entries_that_are_no_pages_take_nothing(gpu):
    x = Append([(70, 70), (20, 2)], 4, 2, 64, 16, BF16, seed=4)
    for b, p, bad in ((0, 1, -1), (0, 4, x.n_pages), (1, 1, -2 ** 31)):
        x.table[b, p] = bad
        x.table_l[b][p] = bad
    f = attn.attn_rope_frequencies(64)
    want = [x.kp.clone(), x.vp.clone()]
    k_out = torch.empty_like(x.k)
    q = x.call(f, k_out=k_out)[0]
    attn.attn_device_status()
    check(q, x.q, None, 0, x.positions(), f)
    for b, (L, n) in enumerate(x.seqs):
        for i in range(n):
            page = x.table_l[b][(L - n + i) // 16]
            if 0 <= page < x.n_pages:
                want[0][page, :, (L - n + i) % 16] = k_out[x.ends[b] + i]
                want[1][page, :, (L - n + i) % 16] = x.v[x.ends[b] + i]
    assert torch.equal(x.kp, want[0]) and torch.equal(x.vp, want[1])


def test_captured_on_a_side_stream(gpu):
    x = Append([(40, 40), (100, 1)], 4, 2, 64, 16, BF16, seed=6)
    f, (wq, wk) = attn.attn_rope_frequencies(64), weights(64, BF16, 7)
    x.call(f, q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = x.call(f, q_weight=wq, k_weight=wk)
    x.lens.copy_(ints([41, 99]))
    want_k, want_v = x.kp.clone(), x.vp.clone()
    g.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [x.kp.clone(), x.vp.clone(), q.clone()]
    x.kp.copy_(want_k), x.vp.copy_(want_v)
    side.wait_stream(torch.cuda.current_stream())
    q2 = x.call(f, q_weight=wq, k_weight=wk, stream=side)
    side.synchronize()
    assert torch.equal(got[0], x.kp) and torch.equal(got[1], x.vp) and torch.equal(got[2], q2)
