"""64-bit reference of attention with an arbitrary visibility mask, with bounds on
what the kernels' arithmetic may be off by (test helper).

A row's weights are p_j = exp(s_j - m), out = sum p_j v_j / sum p_j.  With
A = sum p_j |v_j| / sum p_j and E = max |error of a score|:

* scores: a sum of D products in fp32, each partial sum rounded (or, in the
  tensor cores, cut) to 24 bits, then one product with the scale: E is at most
  (D + 4) u scale max_j sum_d |q_d k_jd|, u = 2^-24 for FMA chains, 2^-23 cut;
* weights: exp turns E into a relative 2 E (numerator and sum), the
  exponential itself is good to 2^-21;
* sums over n keys in fp32: (n + 8) 2^-23;
* bf16: P is rounded to bf16 (half a step, 2^-8 of each weight) and so is the
  result (2^-8 of it).
"""
from __future__ import annotations

import math

import torch


def attend(q, k, v, visible, scale):
    """(out, lse, A, largest sum |q k|) in float64 for q (n, D), k and v (m, D);
    masked values are taken out, not multiplied by zero."""
    q, k, v = q.double(), k.double(), v.double()
    s = torch.where(visible, (torch.nan_to_num(q) @ torch.nan_to_num(k).T) * scale, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.clamp(min=-1e300)[:, None])
    p = torch.where(visible, p, torch.zeros_like(p))
    size = (torch.nan_to_num(q).abs() @ torch.nan_to_num(k).abs().T).max() if k.numel() and q.numel() else torch.zeros(())
    return p @ torch.nan_to_num(v, 0.0, 0.0, 0.0), lse, p @ torch.nan_to_num(v, 0.0, 0.0, 0.0).abs(), float(size)


def bounds(dtype, D, n, scale, size, out, A):
    """(bound on |out error|, bound on |lse error| without the |lse| term)."""
    bf16 = dtype == torch.bfloat16
    E = (D + 4) * (2.0 ** -23 if bf16 else 2.0 ** -24) * scale * size
    rel = 2 * E + 2.0 ** -20 + (n + 8) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    tol = (rel + (half if bf16 else 0.0)) * A
    return tol + (out.abs() + tol) * half + 1e-30, E + 2.0 ** -19 + (n + 8) * 2.0 ** -23


def check(got, out, tol, what=""):
    err = (got.double() - out).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite output"
    assert torch.all(err <= tol), f"{what}: worst excess {(err - tol).max():.3e}, worst error {err.max():.3e}"


def huge_inputs(n_rows, n_keys, D, dtype, seed):
    """q (n_rows, D) and k (n_keys, D) of one nonzero element each, whose scores are exact
    in fp32, of both signs, 2^27 to 2^92 in magnitude and growing from tile to tile of 128
    keys; two scores of a row are equal or differ by 2^-8 of them.  Every fourth row
    is zero."""
    g = torch.Generator().manual_seed(seed)

    def pick(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g)

    j = torch.arange(n_keys)
    b = pick(128, 256, n_keys) * 2.0 ** (20 + (3 * (j // 128)).clamp(max=30) + pick(0, 3, n_keys)) * (2 * pick(0, 2, n_keys) - 1)
    i = torch.arange(n_rows)
    a = 2.0 ** torch.tensor([0.0, 10.0, 32.0, 0.0])[i % 4] * (2 * pick(0, 2, n_rows) - 1) * (i % 4 != 3)
    q, k = torch.zeros(n_rows, D), torch.zeros(n_keys, D)
    q[:, 0], k[:, 0] = a, b
    return q.to(dtype).cuda(), k.to(dtype).cuda()


def check_huge(got, lse, q, k, v, visible, dtype, what=""):
    """Rows of huge_inputs (scale 1): the weights are 1 at the largest score (equal
    scores share it) and underflow elsewhere, so the mean of those values comes out
    of one product, one division and one rounding; a zero row is the mean of all it sees.
    The log-sum-exp is the score through four products rounded to 24 bits."""
    s = torch.where(visible, q.double() @ k.double().T, -math.inf)
    top = (s == s.amax(-1, keepdim=True)) & visible
    n = top.sum(-1, keepdim=True)
    mean, size = top.double() @ v.double() / n, top.double() @ v.double().abs() / n
    half = torch.finfo(dtype).eps / 2
    tol = size * ((n + 8) * 2.0 ** -23) + (mean.abs() + size * 2.0 ** -12) * half + 1e-30
    check(got, mean, tol, what)
    if lse is not None:
        want = s.amax(-1) + torch.log(n[:, 0].double())
        err = (lse.double() - want).abs()
        assert torch.all(err <= want.abs() * 2.0 ** -21 + 2.0 ** -18), f"{what} lse {err.max():.3e}"
