"""The calls of a paged cache used together, as a serving program uses them: prompts come
into pages in chunks, tokens are decoded beside them, sequences fork into beams that share
pages, drafts are cut back, sequences end and new ones take their pages, the pool is moved
together.  A model of each sequence on the side, its keys and values in order, gives
every step's attention in 64 bits, whatever pages they went through."""
from __future__ import annotations

import random

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
import serving_ref as ref

pytestmark = pytest.mark.gpu

LAYERS, H, H_KV, P, M = 2, 8, 2, 16, 20


def ints(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


class Server:
    def __init__(self, dtype, D, n_pages, seed):
        self.dtype, self.D, self.n_pages = dtype, D, n_pages
        self.g = torch.Generator().manual_seed(seed)
        self.kp, self.vp = (torch.full((LAYERS, n_pages, H_KV, P, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.freqs = attn.attn_rope_frequencies(D)
        self.weights = [(1 + 0.2 * torch.randn(D, generator=self.g)).to(dtype).cuda() for _ in range(2)]
        self.table, self.lens = torch.empty(0, M, dtype=torch.int32, device="cuda"), ints([])
        self.seqs = []  # per row and layer: (keys, values) in order

    def step(self, parents, new):
        """Rows go on from their parents (-1: a new sequence) with `new` tokens more (cut back where negative)."""
        old = [len(s[0][0]) for s in self.seqs]
        base = [old[p] if p >= 0 else 0 for p in parents]
        lens = [b + n for b, n in zip(base, new)]
        self.table, self.lens, copies, free = attn.attn_pages_step(
            self.table, self.lens, self.n_pages, P, parents=ints(parents), new_len=ints(lens))
        attn.attn_pages_copy(self.kp, self.vp, copies)
        assert free.item() >= 0 and self.lens.tolist() == lens
        self.seqs = [[(k[:n], v[:n]) for k, v in self.seqs[p]] if p >= 0 else
                     [(torch.empty(0, H_KV, self.D, dtype=self.dtype, device="cuda"),) * 2 for _ in range(LAYERS)]
                     for p, n in zip(parents, lens)]
        tokens = [max(n, 0) for n in new]
        if not sum(tokens):
            return
        cu = ints([sum(tokens[:i]) for i in range(len(tokens) + 1)])
        one_each = all(n == 1 for n in tokens)
        for layer in range(LAYERS):
            qkv = torch.randn(sum(tokens), H + 2 * H_KV, self.D, generator=self.g).to(self.dtype).cuda()
            q, k, v = qkv[:, :H], qkv[:, H:H + H_KV], qkv[:, H + H_KV:]
            kw = dict(cu_seqlens=None if one_each else cu)
            k_out = torch.empty(k.shape, dtype=self.dtype, device="cuda")
            q, _ = attn.attn_rope_append_paged(q, k, v, self.kp[layer], self.vp[layer], self.table, self.freqs, self.lens,
                                               q_weight=self.weights[0], k_weight=self.weights[1], k_out=k_out, **kw)
            out, lse = attn.attn_fwd_paged(q, self.kp[layer], self.vp[layer], self.table, self.lens, return_lse=True, **kw)
            attn.attn_device_status()
            first = 0
            for b, n in enumerate(tokens):
                rows = slice(first, first + n)
                first += n
                ks, vs = self.seqs[b][layer]
                ks, vs = torch.cat((ks, k_out[rows])), torch.cat((vs, v[rows]))
                self.seqs[b][layer] = ks, vs
                if n:
                    self.check(b, layer, q[rows], ks, vs, out[rows], lse[rows])

    def check(self, b, layer, q, k, v, out, lse):
        n, L = q.shape[0], k.shape[0]
        see = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda")[:, None]
        for h in range(H):
            o, l, A, size = ref.attend(q[:, h], k[:, h * H_KV // H], v[:, h * H_KV // H], see, self.D ** -0.5)
            tol, ltol = ref.bounds(self.dtype, self.D, L, self.D ** -0.5, size, o, A)
            ref.check(out[:, h], o, tol, f"row {b} layer {layer} (L {L}, n {n}) head {h}")
            assert torch.all((lse[:, h].double() - l).abs() <= ltol + l.abs() * 2.0 ** -21)

    def compact(self):
        self.table, copies, free = attn.attn_pages_compact(self.table, self.lens, self.n_pages, P)
        attn.attn_pages_copy(self.kp, self.vp, copies)
        held = {p for row, n in zip(self.table.tolist(), self.lens.tolist()) for p in row[:-(-n // P)]}
        assert held == set(range(len(held))) and free.item() == self.n_pages - len(held)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_prompts_beams_drafts_and_ends(gpu, dtype, D):
    s = Server(dtype, D, 60, 1)
    s.step([-1, -1, -1], [70, 5, 33])              # three prompts
    s.step([0, 1, 2], [50, 1, 1])                  # a chunk of the first beside decoding ones
    s.step([0, 1, 2], [1, 1, 1])
    s.step([0, 1, 1, 1, 2], [1, 1, 1, 1, 1])       # the second forks into three beams
    s.step([0, 2, 2, 3, 4], [1, 1, 1, 1, 1])       # two of them go on, one ends
    s.step([0, 1, 2, 3, 4], [7, 7, 7, 7, 7])       # drafts
    s.step([0, 1, 2, 3, 4], [-6, -3, -7, 0, -5])   # some are cut back
    s.step([0, 1, 2, 3, 4], [1, 1, 1, 1, 1])
    s.step([0, 3, -1], [1, 1, 40])                 # others end, a new prompt takes their pages
    s.compact()
    s.step([0, 1, 2], [1, 20, 1])
    s.step([2, 2, 0], [1, 1, 1])
    s.compact()
    s.step([0, 1, 2], [1, 1, 1])


def test_a_random_life(gpu):
    r = random.Random(4)
    s = Server(torch.bfloat16, 64, 200, 2)
    s.step([-1] * 4, [r.randint(1, 60) for _ in range(4)])
    for _ in range(25):
        lens = [len(x[0][0]) for x in s.seqs]
        parents, new = [], []
        for b, L in enumerate(lens):
            if L > 250 or r.random() < 0.1:
                continue
            for _ in range(r.choice((1, 1, 1, 2))):
                parents.append(b)
                new.append(r.choice((1, 1, 1, r.randint(2, 40), -r.randint(0, L))))
        while len(parents) < 3:
            parents.append(-1)
            new.append(r.randint(1, 80))
        s.step(parents[:8], new[:8])
        if r.random() < 0.2:
            s.compact()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_step_captured(gpu, dtype):
    """Table, append and attention of one decode step as a graph; replayed over a growing sequence it walks
    through the pages as separate calls do."""
    D, B, n_pages = 64, 3, 40
    g = torch.Generator().manual_seed(9)
    freqs = attn.attn_rope_frequencies(D)

    def fresh():
        kp, vp = (torch.zeros(n_pages, H_KV, P, D, dtype=dtype, device="cuda") for _ in range(2))
        return kp, vp, torch.full((B, M), -1, dtype=torch.int32, device="cuda"), ints([0] * B)

    qkv = torch.empty(B, H + 2 * H_KV, D, dtype=dtype, device="cuda")

    def step(kp, vp, table, lens):
        t, n, copies, free = attn.attn_pages_step(table, lens, n_pages, P, new_len=lens + 1)
        attn.attn_pages_copy(kp, vp, copies)
        table.copy_(t), lens.copy_(n)
        q = attn.attn_rope_append_paged(qkv[:, :H], qkv[:, H:H + H_KV], qkv[:, H + H_KV:], kp, vp, table, freqs, lens)
        return attn.attn_fwd_paged(q, kp, vp, table, lens)

    a, b = fresh(), fresh()
    qkv.copy_(torch.randn(qkv.shape, generator=g))
    step(*fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*a)
    for x, y in zip(a, fresh()):
        x.copy_(y)
    for _ in range(37):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        graph.replay()
        want = step(*b)
        torch.cuda.synchronize()
        attn.attn_device_status()
        assert torch.equal(out, want)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and a[3].tolist() == [37] * B
