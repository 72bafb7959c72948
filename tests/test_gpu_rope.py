"""GPU parity tests of attn_rope and attn_rope_append against the definition in
64 bits (complex turns on the CPU).

Tolerance.  The kernel's angle is off by at most 2^-25 half turns (the
fraction of a turn rounded to fp32) plus terms below 1e-8, which is 1.0e-7
radians; sincospif is good to 2 ulp, 1.2e-7; so cos and sin are off by at most
2.2e-7, and mscale adds 2^-24 = 6e-8.  Each output is a sum of two products,
three roundings of at most 2^-24 each: 1.8e-7 of |a| + |b|.  Together less than
5e-7 mscale (|a| + |b|), and the one rounding to the output type: 2^-8 of the
value for bf16.
"""
from __future__ import annotations

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def turned(x, positions, freqs, interleaved=False, inverse=False, mscale=1.0):
    """(the turned rows in 64 bits, |a| + |b| of each element's pair)."""
    x = x.detach().cpu().double()
    r = 2 * freqs.numel()
    angle = positions.cpu().double()[:, None, None] * freqs
    if inverse:
        angle = -angle
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    ra, rb = mscale * (a * angle.cos() - b * angle.sin()), mscale * (b * angle.cos() + a * angle.sin())
    out, size = x.clone(), torch.zeros_like(x)
    if interleaved:
        out[..., 0:r:2], out[..., 1:r:2] = ra, rb
        size[..., 0:r:2] = size[..., 1:r:2] = a.abs() + b.abs()
    else:
        out[..., :r // 2], out[..., r // 2:r] = ra, rb
        size[..., :r // 2] = size[..., r // 2:r] = a.abs() + b.abs()
    return out, size


def check(got, ref, size, mscale=1.0, what=""):
    tol = 5e-7 * abs(mscale) * size
    if got.dtype == BF16:
        tol = tol + (ref.abs() + tol) * (torch.finfo(BF16).eps / 2)
    err = (got.cpu().double() - ref).abs()
    assert torch.all(err <= tol), f"{what}: worst excess {(err - tol).max():.3e}"


def rows(T, heads, D, seed, dtype):
    return wl.random_tensors((T, heads, D), seed, dtype=dtype, count=1)[0]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 64), (128, 36), (128, 2), (128, 0), (64, 64), (64, 48), (64, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(gpu, dtype, D, rd, interleaved, inverse):
    T, H, H_kv = 37, 6, 2
    q, k = rows(T, H, D, 1, dtype), rows(T, H_kv, D, 2, dtype)
    pos = torch.randint(0, 1 << 21, (T,), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    pos[:4] = ints([0, 1, -5, 131071])
    f = attn.attn_rope_frequencies(rd)
    qo, ko = attn.attn_rope(q, k, pos, f, interleaved=interleaved, inverse=inverse, mscale=1.25)
    for x, got in ((q, qo), (k, ko)):
        ref, size = turned(x, pos, f, interleaved, inverse, 1.25)
        check(got, ref, size, 1.25, f"D={D} rd={rd}")
        assert torch.equal(got[..., rd:], x[..., rd:])


@pytest.mark.parametrize("T", [1, 2, 303, 1217, 5000])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (32, 8), (5, 0)])
def test_rope_sizes(gpu, T, H, H_kv):
    q = rows(T, H, 128, 4, BF16)
    k = rows(T, H_kv, 128, 5, BF16) if H_kv else None
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    f = attn.attn_rope_frequencies(128, theta=500000.0)
    out = attn.attn_rope(q, k, pos, f)
    for x, got in zip((q, k), out if H_kv else (out,)):
        ref, size = turned(x, pos, f)
        check(got, ref, size)


def test_far_positions_keep_their_angle(gpu):
    """At 2^31 - 1 a product in fp32 would be off by whole turns.  The reference
    angle, a 64-bit product of up to 2^31, is off by up to 2^-23 radians, and the
    kernel's w / 2 pi, rounded to 53 bits twice, by 2^-22: 3.6e-7 more per
    element of the pair, covered by twice the tolerance."""
    q = rows(3, 2, 64, 6, F32)
    pos = ints([2147483647, -2147483648, 2000000011])
    f = attn.attn_rope_frequencies(64)
    ref, size = turned(q, pos, f)
    check(attn.attn_rope(q, None, pos, f), ref, 2 * size)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_slices_of_one_projection(gpu, dtype, interleaved):
    T, H, H_kv, D, rd = 50, 4, 2, 64, 32
    qkv = rows(T, H + 2 * H_kv, D, 7, dtype)
    keep = qkv.clone()
    q, k = qkv[:, :H], qkv[:, H:H + H_kv]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = attn.attn_rope_frequencies(rd)
    out = attn.attn_rope(q, k, pos, f, q_out=q, k_out=k, interleaved=interleaved)
    assert out[0].data_ptr() == q.data_ptr() and out[1].data_ptr() == k.data_ptr()
    ref, size = turned(keep[:, :H + H_kv], pos, f, interleaved)
    check(qkv[:, :H + H_kv], ref, size)
    assert torch.equal(qkv[:, H + H_kv:], keep[:, H + H_kv:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_strides_and_addresses(gpu, dtype):
    """Rows that start at single elements, head-major rows, odd strides."""
    T, H, D, rd = 20, 3, 64, 64
    f = attn.attn_rope_frequencies(rd)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 100
    base = rows(1, 1, T * (H * 71 + 5) + 3, 8, dtype).flatten()
    q = base[3:].as_strided((T, H, D), (H * 71 + 5, 71, 1))
    ref, size = turned(q, pos, f)
    check(attn.attn_rope(q, None, pos, f), ref, size)
    hm = rows(H, T, D, 9, dtype).transpose(0, 1)  # (T, H, D) over a head-major buffer
    out = torch.empty((H, T, D), dtype=dtype, device="cuda").transpose(0, 1)
    ref, size = turned(hm, pos, f)
    check(attn.attn_rope(hm, None, pos, f, q_out=out), ref, size)


def test_inverse_is_the_gradient(gpu):
    """<R x, g> and <x, R^T g> agree, and a difference along a direction is R of it."""
    T, H, D = 40, 3, 128
    x, g, d = (rows(T, H, D, s, F32) for s in (10, 11, 12))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 31
    f = attn.attn_rope_frequencies(96)
    turn = lambda y, inv=False: attn.attn_rope(y, None, pos, f, inverse=inv, mscale=0.75).double()  # noqa: E731
    grad = turn(g, True)
    ref, size = turned(g, pos, f, False, True, 0.75)
    check(grad.float(), ref, size, 0.75)
    # loss = <R x, g>; its difference along d, with a step of 1 (the loss is linear)
    num = ((turn(x + d) - turn(x)) * g.double()).sum().item()
    ana = (grad * d.double()).sum().item()
    # each of 15360 terms is off by at most about 5e-7 * 2 * |x| |g|: they add up like sqrt(n)
    scale = (x.double().abs() + d.double().abs()).max().item() * g.double().abs().max().item()
    assert abs(num - ana) <= 15360 ** 0.5 * 2e-6 * 3 * scale
    # turned forth and back: the rows themselves, times mscale^2
    back = turn(turn(x).float(), True)
    ref, size = turned(x, pos, f)
    assert torch.all((back.cpu()[..., :96] - 0.5625 * x.cpu().double()[..., :96]).abs()
                     <= 4 * 5e-7 * 0.75 * (size[..., :96] + 1e-30) * 1.5)


def _append_case(lens, past, Skv, H, H_kv, D, rd, dtype, interleaved=False, positions=None, lead=0, trail=0, k_out=False,
                 seed=20):
    B, T = len(lens), sum(lens) + lead + trail
    cu = [lead + sum(lens[:i]) for i in range(B + 1)]
    qkv = rows(max(T, 1), H + 2 * H_kv, D, seed, dtype)[:T]
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), seed + 1, dtype=dtype, count=2)
    want_k, want_v = kc.cpu().double(), vc.cpu().double()
    size_k = torch.zeros_like(want_k)
    cl = [p + n for p, n in zip(past, lens)]
    f = attn.attn_rope_frequencies(rd)
    q_out = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    ko = torch.full((T, H_kv, D), 7.0, dtype=dtype, device="cuda") if k_out else None
    want_q, size_q = torch.full((T, H, D), 7.0, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    want_ko, size_ko = want_q[:, :H_kv].clone(), size_q[:, :H_kv].clone()
    for b, n in enumerate(lens):
        for i in range(n):
            t, L = cu[b] + i, min(max(cl[b], 0), Skv)
            row = L - n + i
            p = torch.tensor([positions[t] if positions is not None else row])
            want_q[t], size_q[t] = (z[0] for z in turned(q[t:t + 1], p, f, interleaved))
            kk, ks = (z[0] for z in turned(k[t:t + 1], p, f, interleaved))
            want_ko[t], size_ko[t] = kk, ks
            if row >= 0:
                want_k[b, :, row], size_k[b, :, row] = kk, ks
                want_v[b, :, row] = v[t].cpu().double()
    pos = ints(positions) if positions is not None else None
    out = attn.attn_rope_append(q, k, v, kc, vc, f, cu_seqlens=ints(cu), cache_len=ints(cl), positions=pos, q_out=q_out,
                                k_out=ko, interleaved=interleaved)
    torch.cuda.synchronize()
    got_q = out[0] if k_out else out
    assert got_q.data_ptr() == q_out.data_ptr()
    check(got_q, want_q, size_q, what="q")
    check(kc, want_k, size_k, what="kcache")
    assert torch.equal(vc.cpu().double(), want_v)
    if k_out:
        check(ko, want_ko, size_ko, what="k_out")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rd", [(128, 128), (64, 20)])
@pytest.mark.parametrize("k_out", [False, True])
def test_append_ragged(gpu, dtype, D, rd, k_out):
    _append_case([3, 0, 1, 40, 7], [0, 5, 63, 10, 100], 128, 4, 2, D, rd, dtype, k_out=k_out, lead=2, trail=3)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_cuts_at_the_cache(gpu, interleaved):
    """Lengths past the capacity are clamped: the last tokens end at the last
    row and tokens before row 0 are turned, not cached."""
    _append_case([6, 4, 9], [0, 30, -4], 8, 2, 1, 64, 64, BF16, interleaved=interleaved)


def test_append_positions_of_a_tree(gpu):
    lens = [5, 5]
    _append_case(lens, [11, 3], 32, 4, 4, 128, 128, BF16, positions=[11, 12, 12, 13, 13, 3, 4, 5, 5, 4])


def test_append_many_sequences(gpu):
    lens = [(7 * i) % 4 for i in range(1100)]
    _append_case(lens, [i % 5 for i in range(1100)], 16, 1, 1, 64, 32, F32)


def test_append_one_token_each_without_cu_seqlens(gpu):
    B, H, H_kv, D, Skv = 9, 8, 2, 128, 40
    q, k, v = rows(B, H, D, 30, BF16), rows(B, H_kv, D, 31, BF16), rows(B, H_kv, D, 32, BF16)
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 33, count=2)
    kc2, vc2 = kc.clone(), vc.clone()
    f = attn.attn_rope_frequencies(D)
    cl = ints(list(range(1, B + 1)))
    a = attn.attn_rope_append(q, k, v, kc, vc, f, cache_len=cl)
    b = attn.attn_rope_append(q, k, v, kc2, vc2, f, cache_len=cl, cu_seqlens=torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    # no cache_len: the whole capacity counts, the token goes to the last row
    attn.attn_rope_append(q, k, v, kc, vc, f)
    assert torch.equal(vc[:, :, -1], v)


def test_append_into_a_cache_past_2_gi_elements(gpu):
    """Row offsets pass 32 bits: 2.2e9 elements in one cache."""
    B, H_kv, Skv, D = 2, 8, 1 << 20, 128
    kc = torch.zeros((B, H_kv, Skv, D), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v = rows(4, 8, D, 34, BF16), rows(4, H_kv, D, 35, BF16), rows(4, H_kv, D, 36, BF16)
    f = attn.attn_rope_frequencies(D)
    attn.attn_rope_append(q, k, v, kc, vc, f, cache_len=ints([2, Skv]))
    assert torch.equal(vc[0, :, :2], v[:2].transpose(0, 1)) and torch.equal(vc[1, :, -2:], v[2:].transpose(0, 1))
    assert torch.count_nonzero(vc[1, :, :-2]) == 0 and torch.count_nonzero(vc[0, :, 2:]) == 0
    ref, size = turned(k[2:], torch.tensor([Skv - 2, Skv - 1]), f)
    check(kc[1, :, -2:].transpose(0, 1), ref, size)


def test_malformed_lengths_stay_inside(gpu):
    """cu_seqlens that decrease or leave [0, T] touch nothing outside the tensors:
    tokens without a sequence stay as they were."""
    T, H, D, Skv = 12, 2, 64, 16
    q, k, v = rows(T, H, D, 37, BF16), rows(T, H, D, 38, BF16), rows(T, H, D, 39, BF16)
    f = attn.attn_rope_frequencies(D)
    for cu in ([5, 3, 100, 12], [-50, -20, -3, -1], [2000000000, -2000000000, 7, 3], [0, 4, 4, 4]):
        kc, vc = wl.random_tensors((3, H, Skv, D), 40, count=2)
        q_out = torch.zeros_like(q)
        attn.attn_rope_append(q, k, v, kc, vc, f, cu_seqlens=ints(cu), cache_len=ints([4, 400, -7]), q_out=q_out)
        torch.cuda.synchronize()
        assert torch.isfinite(kc.float()).all() and torch.isfinite(q_out.float()).all()
    assert torch.count_nonzero(q_out[4:]) == 0


def test_captured_and_on_another_stream(gpu):
    T, H, H_kv, D, B, Skv = 30, 4, 2, 128, 3, 64
    q, k, v = rows(T, H, D, 41, BF16), rows(T, H_kv, D, 42, BF16), rows(T, H_kv, D, 43, BF16)
    kc, vc = wl.random_tensors((B, H_kv, Skv, D), 44, count=2)
    f = attn.attn_rope_frequencies(D)
    cl = ints([10, 20, 64])
    q_out = torch.empty_like(q)
    kc0, vc0 = kc.clone(), vc.clone()
    ref = attn.attn_rope_append(q, k, v, kc0, vc0, f, cache_len=cl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        attn.attn_rope_append(q, k, v, kc, vc, f, cache_len=cl, q_out=q_out)
    f.zero_()  # the captured call keeps its values
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, ref) and torch.equal(kc, kc0) and torch.equal(vc, vc0)
    f = attn.attn_rope_frequencies(D)
    q_out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    attn.attn_rope_append(q, k, v, kc, vc, f, cache_len=cl, q_out=q_out, stream=s)
    s.synchronize()
    assert torch.equal(q_out, ref)


def test_gpu_refusals(gpu):
    q, k = rows(4, 2, 64, 50, BF16), rows(4, 2, 64, 51, BF16)
    pos, f = ints([0, 1, 2, 3]), attn.attn_rope_frequencies(64)
    with pytest.raises(TypeError):
        attn.attn_rope(q, k.float(), pos, f)
    with pytest.raises(TypeError):
        attn.attn_rope(q.half(), None, pos, f)
    for args in ((q, k[:3], pos, f), (q, k, pos[:3], f), (q, k, pos.long(), f), (q, k, None, f), (q.transpose(1, 2), None, pos, f),
                 (q, k, pos, f.cuda())):
        with pytest.raises(ValueError):
            attn.attn_rope(*args)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_rope(q, k, pos, f, q_out=k)
    assert e.value.code == attn.ATTN_EINVAL
    kc = torch.zeros(3, 2, 8, 64, dtype=BF16, device="cuda")
    with pytest.raises(attn.AttnError):  # 4 tokens for 3 sequences without cu_seqlens
        attn.attn_rope_append(q, k, k.clone(), kc, kc.clone(), f)


def test_far_positions_and_negative_frequencies(gpu):
    """Positions to the ends of int32 and frequencies of both signs, angles from exact
    integers (w as a ratio of integers, 2 pi to 40 digits): the usual tolerance."""
    two_pi = 62831853071795864769252867665590057683943   # 1e40 times
    q = rows(4, 3, 64, 30, F32)
    positions = [2147483647, -2147483648, 2147480009, -1999999999]
    for sign in (1, -1):
        f = sign * attn.attn_rope_frequencies(64)
        angle = torch.empty(4, 32, dtype=torch.float64)
        for i, n in enumerate(positions):
            for p, w in enumerate(f.tolist()):
                top, bottom = w.as_integer_ratio()
                left = (n * top * 10 ** 40) % (two_pi * bottom)   # what whole turns leave over
                angle[i, p] = left / (bottom * 10 ** 40)
        a, b = q.cpu().double()[..., :32], q.cpu().double()[..., 32:]
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        size = torch.cat([a.abs() + b.abs()] * 2, -1)
        check(attn.attn_rope(q, None, ints(positions), f), torch.cat((a * c - b * s, b * c + a * s), -1), size, what=f"{sign}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_to_a_cache_of_no_rows(gpu, dtype):
    """Every token is turned, none cached, as attn_decode_tree takes such a cache."""
    T, H, H_kv, D = 6, 4, 2, 64
    q, k, v = rows(T, H, D, 37, dtype), rows(T, H_kv, D, 38, dtype), rows(T, H_kv, D, 39, dtype)
    none = torch.empty((2, H_kv, 0, D), dtype=dtype, device="cuda")
    f = attn.attn_rope_frequencies(D)
    pos = ints([0, 3, 70000, -4, 9, 1])
    qo, ko = attn.attn_rope_append(q, k, v, none, none.clone(), f, positions=pos, k_out=torch.empty_like(k))
    for x, got in ((q, qo), (k, ko)):
        check(got, *turned(x, pos, f))
    qo = attn.attn_rope_append(q, k, v, none, none.clone(), f, cu_seqlens=ints([0, 4, 6]))
    # token i of n goes to row i - n of no cache, which is its position
    check(qo, *turned(q, torch.tensor([-4, -3, -2, -1, -2, -1]), f))
