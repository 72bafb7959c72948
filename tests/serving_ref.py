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
