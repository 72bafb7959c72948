"""The serving calls used together, as a program that drafts and verifies uses
them: packed prompts are turned and appended to the cache and attend to
themselves, a token is decoded, a tree of drafts is appended at positions by
depth and attends to the cache, an accepted branch is moved into place and the
next token is decoded.  Every step is checked against the definition in 64 bits
on what the step before left (the rotation itself is held in test_gpu_rope.py),
eagerly and as one captured graph."""
from __future__ import annotations

import math

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import workloads as wl
import serving_ref as ref

pytestmark = pytest.mark.gpu

LENS = [70, 1, 333]
PARENTS = [-1, 0, 0, 1, 3, 2, -1]     # 0-1-3-4 is the branch taken; 6 a second root
BRANCH = [0, 1, 3, 4]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def depth(t):
    return 0 if PARENTS[t] < 0 else 1 + depth(PARENTS[t])


def check_rows(q, kc, vc, b, h, G, visible_rows, out, what):
    """out row of query row q over the given cache rows of sequence b."""
    D = q.shape[-1]
    k, v = kc[b, h // G, visible_rows], vc[b, h // G, visible_rows]
    see = torch.ones(1, len(visible_rows), dtype=torch.bool, device="cuda")
    o, _, A, size = ref.attend(q[None], k, v, see, D ** -0.5)
    tol, _ = ref.bounds(q.dtype, D, len(visible_rows), D ** -0.5, size, o, A)
    ref.check(out[None], o, tol, what)


class Run:
    def __init__(self, dtype, D, H=8, H_kv=2, Skv=400, seed=1):
        self.dtype, self.D, self.H, self.H_kv, self.G = dtype, D, H, H_kv, H // H_kv
        B, n = len(LENS), len(PARENTS)
        new = lambda T, s: wl.random_tensors((T, H + 2 * H_kv, D), s, dtype=dtype, count=1)[0]  # noqa: E731
        self.prompt, self.tok1, self.draft, self.tok2 = new(sum(LENS), seed), new(B, seed + 1), new(B * n, seed + 2), new(B, seed + 3)
        self.kc, self.vc = (torch.full((B, H_kv, Skv, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
        self.freqs = attn.attn_rope_frequencies(D // 2, scaling="wavelength", factor=8.0)
        self.cu = ints([sum(LENS[:b]) for b in range(B + 1)])
        self.len0 = ints(LENS)
        self.len1, self.len2, self.len3 = ints([x + 1 for x in LENS]), ints([x + 1 + n for x in LENS]), ints([x + 2 + len(BRANCH) for x in LENS])
        self.pos = ints([x + 1 + depth(t) for x in LENS for t in range(n)])
        self.parents = ints(PARENTS)
        base = torch.tensor([x + 1 for x in LENS], device="cuda")
        self.src = base[:, None] + torch.tensor(BRANCH, device="cuda")
        self.dst = base[:, None] + torch.arange(len(BRANCH), device="cuda")

    def split(self, x):
        return x[:, :self.H], x[:, self.H:self.H + self.H_kv], x[:, self.H + self.H_kv:]

    def steps(self):
        B, n = len(LENS), len(PARENTS)
        kw = dict(freqs=self.freqs, interleaved=True)
        q, k, v = self.split(self.prompt)
        self.k0 = torch.empty(k.shape, dtype=k.dtype, device="cuda")
        self.q0, _ = attn.attn_rope_append(q, k, v, self.kc, self.vc, cu_seqlens=self.cu, cache_len=self.len0, k_out=self.k0, **kw)
        self.out0 = attn.attn_fwd_packed(self.q0, self.k0, v, self.cu, causal=True)
        self.q1 = attn.attn_rope_append(*self.split(self.tok1), self.kc, self.vc, cache_len=self.len1, **kw)
        self.out1 = attn.attn_decode(self.q1, self.kc, self.vc, kv_len=self.len1)
        self.q2 = attn.attn_rope_append(*self.split(self.draft), self.kc, self.vc, cache_len=self.len2, positions=self.pos, **kw)
        self.out2 = attn.attn_decode_tree(self.q2.view(B, n, self.H, self.D).transpose(1, 2), self.kc, self.vc, self.parents,
                                          cache_len=self.len2)
        self.kc2, self.vc2 = self.kc.clone(), self.vc.clone()
        b = torch.arange(B, device="cuda")[:, None]
        for c in (self.kc, self.vc):
            c[b, :, self.dst] = c[b, :, self.src]
        self.q3 = attn.attn_rope_append(*self.split(self.tok2), self.kc, self.vc, cache_len=self.len3, **kw)
        # bf16 decode reads whole tiles: what lies past the length must be finite there
        self.kc3, self.vc3 = self.kc.nan_to_num(), self.vc.nan_to_num()
        self.out3 = attn.attn_decode(self.q3, self.kc3, self.vc3, kv_len=self.len3)

    def outputs(self):
        return [self.out0, self.out1, self.out2, self.out3]


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_draft_and_verify(gpu, dtype, D):
    r = Run(dtype, D)
    r.kc.nan_to_num_(), r.vc.nan_to_num_()
    r.steps()
    attn.attn_device_status()
    n = len(PARENTS)
    first = 0
    for b, L in enumerate(LENS):
        rows = slice(first, first + L)
        # the appended rows are the turned keys and the values
        assert torch.equal(r.kc2[b, :, :L], r.k0[rows].transpose(0, 1))
        assert torch.equal(r.vc2[b, :, :L], r.split(r.prompt)[2][rows].transpose(0, 1))
        i = torch.arange(L, device="cuda")
        for h in range(r.H):
            o, _, A, size = ref.attend(r.q0[rows, h], r.k0[rows, h // r.G], r.split(r.prompt)[2][rows, h // r.G],
                                       i[:, None] >= i, D ** -0.5)
            tol, _ = ref.bounds(dtype, D, L, D ** -0.5, size, o, A)
            ref.check(r.out0[rows, h], o, tol, f"prompt {b}")
            check_rows(r.q1[b, h], r.kc2, r.vc2, b, h, r.G, list(range(L + 1)), r.out1[b, h], "token after the prompt")
            for t in range(n):
                path, j = [], t
                while j >= 0:
                    path.append(L + 1 + j)
                    j = PARENTS[j]
                check_rows(r.q2[b * n + t, h], r.kc2, r.vc2, b, h, r.G, list(range(L + 1)) + path, r.out2[b, h, t], f"draft {t}")
            check_rows(r.q3[b, h], r.kc3, r.vc3, b, h, r.G, list(range(L + 2 + len(BRANCH))), r.out3[b, h], "token after the branch")
        # the branch's rows moved up keep their positions: the token after it is turned by its row
        for d, t in enumerate(BRANCH):
            assert torch.equal(r.kc3[b, :, L + 1 + d], r.kc2[b, :, L + 1 + t])
            assert int(r.pos[b * n + t]) == L + 1 + d
        first += L


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_run_captured(gpu, dtype):
    """The whole run as one graph, replayed on new prompts and a cleared cache."""
    r = Run(dtype, 128, seed=20)
    r.kc.nan_to_num_(), r.vc.nan_to_num_()
    r.steps()  # sizes the decode workspace
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.steps()
    for seed in (30, 40):
        fresh = Run(dtype, 128, seed=seed)
        fresh.kc.nan_to_num_(), fresh.vc.nan_to_num_()
        for name in ("prompt", "tok1", "draft", "tok2", "kc", "vc"):
            getattr(r, name).copy_(getattr(fresh, name))
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in r.outputs()]
        fresh.steps()
        torch.cuda.synchronize()
        attn.attn_device_status()
        for a, b in zip(got, fresh.outputs()):
            assert torch.equal(a, b)


def test_a_cache_of_nan_hurts_no_draft(gpu):
    """The tree call over a cache that was never written past the sequences."""
    r = Run(torch.bfloat16, 128, seed=50)
    clean = Run(torch.bfloat16, 128, seed=50)
    clean.kc.nan_to_num_(), clean.vc.nan_to_num_()
    for x in (r, clean):
        q, k, v = x.split(x.prompt)
        attn.attn_rope_append(q, k, v, x.kc, x.vc, x.freqs, cu_seqlens=x.cu, cache_len=x.len0)
        attn.attn_rope_append(*x.split(x.tok1), x.kc, x.vc, x.freqs, cache_len=x.len1)
        q2 = attn.attn_rope_append(*x.split(x.draft), x.kc, x.vc, x.freqs, cache_len=x.len2, positions=x.pos)
        x.out = attn.attn_decode_tree(q2.view(len(LENS), len(PARENTS), x.H, x.D).transpose(1, 2), x.kc, x.vc, x.parents,
                                      cache_len=x.len2)
    attn.attn_device_status()
    assert torch.isfinite(r.out.float()).all() and torch.equal(r.out, clean.out)
