"""Host-side tests of attn_fwd_packed and attn_decode_tree: refusals before any
CUDA call (the fake addresses are never dereferenced) and workspace sizes."""
from __future__ import annotations

import ctypes

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn

A = [ctypes.c_void_p(0x1000000000 * (i + 1)) for i in range(10)]
I, U, OK = attn.ATTN_EINVAL, attn.ATTN_EUNSUPPORTED, attn.ATTN_OK
BF, F32 = attn.ATTN_BF16, attn.ATTN_F32


def _st(*v):
    return (ctypes.c_longlong * len(v))(*v)


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def packed(lib, q=A[0], k=A[1], v=A[2], o=A[3], lse=None, T=100, H=4, H_kv=2, D=128, st=None, cu=A[5], n=3, scale=0.1,
           causal=1, dtype=BF, ws=A[6], nb=1 << 20):
    return lib.attn_fwd_packed(q, k, v, o, lse, T, H, H_kv, D, st, cu, n, scale, causal, dtype, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(o=None), I), (dict(cu=None), I), (dict(T=-1), I),
    (dict(n=-1), I), (dict(H=0), I), (dict(H_kv=0), I), (dict(H_kv=3), I), (dict(D=0), I), (dict(D=96), U), (dict(D=256), U),
    (dict(dtype=2), I), (dict(scale=float("nan")), I), (dict(scale=-0.5), I), (dict(scale=float("inf")), I), (dict(causal=2), I),
    (dict(q=off(A[0], 8)), I), (dict(cu=off(A[5], 2)), I), (dict(lse=off(A[7], 1)), I),
    (dict(o=A[0]), I), (dict(o=off(A[1], 256)), I), (dict(lse=A[2]), I),
    (dict(st=_st(512, 128, 256, 128, 256, 128, 516, 128)), I),        # out rows 8 bytes off
    (dict(st=_st(512, 120, 256, 128, 256, 128, 512, 128)), I),        # q's heads overlap
    (dict(st=_st(512, 128, 0, 128, 256, 128, 512, 128)), I),          # k broadcast over tokens
    (dict(st=_st(512, 128, -256, 128, 256, 128, 512, 128)), I),
    (dict(st=_st(1 << 40, 128, 256, 128, 256, 128, 512, 128)), I),
    (dict(st=_st(512, 128, 256, 128, (1 << 63) - 16, 128, 512, 128)), I), (dict(st=_st(512, 128, 256, 1 << 56, 256, 128, 512, 128)), I),
    (dict(ws=None), I), (dict(nb=16), I), (dict(ws=off(A[6], 8)), I), (dict(ws=A[3]), I), (dict(ws=A[5]), I),
    (dict(T=2000000000, H=2000, H_kv=1000, nb=1 << 40, o=ctypes.c_void_p(1 << 61), k=ctypes.c_void_p(1 << 60),
          v=ctypes.c_void_p(3 << 59)), I),                            # too many tiles
    (dict(dtype=F32, T=2000000000, H=64, H_kv=64, k=ctypes.c_void_p(1 << 60), v=ctypes.c_void_p(3 << 59),
          o=ctypes.c_void_p(1 << 61)), I),
])
def test_packed_rejects_bad_arguments(attn_lib, kw, code):
    assert packed(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_slices_of_one_projection_do_not_overlap(attn_lib):
    """q, k, v and out as columns of one matrix pass the overlap check (and then
    fail on the missing workspace, before any CUDA call)."""
    row = 4 + 2 + 2 + 4
    st = _st(*(row * 128, 128) * 4)
    kw = dict(q=A[0], k=off(A[0], 4 * 256), v=off(A[0], 6 * 256), o=off(A[0], 8 * 256), st=st, ws=None)
    assert packed(attn_lib, **kw) == I and "workspace" in attn.attn_last_error()
    kw["o"] = off(A[0], 7 * 256)  # one column early: v's last head
    assert packed(attn_lib, **kw) == I and "out overlaps v" in attn.attn_last_error()


def tree(lib, q=A[0], k=A[1], v=A[2], o=A[3], B=2, H=4, H_kv=2, T=8, Skv=200, D=64, st=None, par=A[5], ps=8, cl=A[7],
         dl=A[8], scale=0.1, dtype=BF, ws=A[6], nb=1 << 34):
    return lib.attn_decode_tree(q, k, v, o, B, H, H_kv, T, Skv, D, st, par, ps, cl, dl, scale, dtype, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(o=None), I), (dict(par=None), I), (dict(B=0), I),
    (dict(H=0), I), (dict(H_kv=3), I), (dict(H_kv=0), I), (dict(T=-1), I), (dict(T=129), U), (dict(Skv=-1), I), (dict(D=0), I),
    (dict(D=32), U), (dict(ps=7), I), (dict(ps=-8), I), (dict(dtype=9), I), (dict(scale=float("nan")), I), (dict(scale=-1.0), I),
    (dict(k=off(A[1], 8)), I), (dict(par=off(A[5], 1)), I), (dict(cl=off(A[7], 2)), I), (dict(o=A[0]), I), (dict(o=A[2]), I),
    (dict(st=_st(2048, 512, 64, 2048, 512, 60)), I),        # strides not of 16 bytes
    (dict(st=_st(2048, 512, 64, 2048, 512, 0)), I),         # every token of out in one row
    (dict(st=_st(2048, 512, 64, 1024, 512, 64)), I),        # sequences of out overlap
    (dict(st=_st(-2048, 512, 64, 2048, 512, 64)), I),
    (dict(st=_st(1 << 62, 512, 64, 2048, 512, 64)), I), (dict(st=_st(2048, 512, 64, 1 << 55, 512, 64), B=1 << 20), I),
    (dict(ws=None), I), (dict(nb=100), I), (dict(ws=A[1]), I), (dict(ws=off(A[6], 4)), I),
    (dict(dtype=F32, Skv=60000, ws=None), I),
    (dict(B=70000, H=512, H_kv=512, T=128), I),             # 2^31 rows and more
])
def test_tree_rejects_bad_arguments(attn_lib, kw, code):
    assert tree(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_empty_calls_are_no_ops(attn_lib):
    assert packed(attn_lib, T=0) == OK and packed(attn_lib, n=0) == OK and tree(attn_lib, T=0) == OK
    assert attn.attn_last_error() == ""


def test_workspace_sizes(attn_lib):
    w = attn_lib.attn_fwd_packed_workspace
    assert w(1000, 7, 4, 2, F32) == 0
    assert w(1000, 7, 4, 2, BF) == 16 * (1 + 1000 // 128 + 7)   # an even group: one query tile a unit
    assert w(1000, 7, 4, 4, BF) == 16 * (1 + 1000 // 256 + 7)   # else two
    for bad in ((-1, 1, 4, 2, BF), (1, -1, 4, 2, BF), (1, 1, 4, 3, BF), (1, 1, 4, 2, 5)):
        assert w(*bad) == I
    t = attn_lib.attn_decode_tree_workspace
    assert t(1, 4, 2, 0, 100, 64, BF) == 0 and t(1, 4, 2, 8, 0, 64, BF) == 0
    assert t(1, 4, 2, 8, 64, 64, F32) == 0                      # one split
    assert t(1, 4, 2, 8, 100000, 64, F32) > 0 and t(1, 4, 2, 8, 64, 128, BF) > 0
    for bad in ((0, 4, 2, 8, 64, 64, BF), (1, 4, 2, 129, 64, 64, BF), (1, 4, 2, 8, 64, 96, BF), (1, 4, 2, 8, -1, 64, BF)):
        assert t(*bad) == I


def test_plan_list_holds_every_unit():
    """The workspace's bound on the number of tile units, T / unit + sequences."""
    import random
    r = random.Random(3)
    for _ in range(2000):
        unit = r.choice((128, 256))
        lens = [r.choice((0, 1, unit - 1, unit, unit + 1, r.randint(0, 5000))) for _ in range(r.randint(1, 60))]
        assert sum(-(-n // unit) for n in lens) <= sum(lens) // unit + len(lens)


def test_binding_refuses_cpu_tensors(attn_lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.attn_fwd_packed(x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        attn.attn_decode_tree(x[None], x[None], x[None], torch.zeros(2, dtype=torch.int32))


def test_tree_keys_are_counted_in_32_bits(attn_lib):
    """Caches whose last tile or split ends past 2^31 keys are refused on the host."""
    w = attn_lib.attn_decode_tree_workspace
    for dtype, most in ((BF, 0x7fffff00), (F32, 0x40000000)):
        assert w(1, 1, 1, 8, most, 64, dtype) >= 0
        for Skv in (most + 1, 0x7fffffff):
            assert w(1, 1, 1, 8, Skv, 64, dtype) == I
            assert tree(attn_lib, B=1, H=1, H_kv=1, Skv=Skv, o=ctypes.c_void_p(1 << 60), v=ctypes.c_void_p(1 << 59),
                        ws=ctypes.c_void_p(1 << 58), nb=1 << 50, dtype=dtype) == I
            assert "too large" in attn.attn_last_error()
