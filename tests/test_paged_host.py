"""Host-side tests of the calls of a paged cache: refusals before any CUDA call (the fake
addresses are never dereferenced), workspace sizes, and what the binding leaves to the
checked path."""
from __future__ import annotations

import ctypes

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn

A = [ctypes.c_void_p(0x1000000000 * (i + 1)) for i in range(16)]
I, U, OK = attn.ATTN_EINVAL, attn.ATTN_EUNSUPPORTED, attn.ATTN_OK
BF, F32 = attn.ATTN_BF16, attn.ATTN_F32


def _st(*v):
    return (ctypes.c_longlong * len(v))(*v)


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def paged(lib, q=A[0], k=A[1], v=A[2], o=A[3], lse=None, T=100, H=4, H_kv=2, D=128, st=None, n_pages=100, P=16, table=A[5],
          M=20, ts=20, cu=A[6], cl=A[7], n=3, scale=0.1, dtype=BF, ws=A[8], nb=1 << 34):
    return lib.attn_fwd_paged(q, k, v, o, lse, T, H, H_kv, D, st, n_pages, P, table, M, ts, cu, cl, n, scale, dtype, ws, nb, None)


PAGES = (2 * 16 * 128, 16 * 128, 128) * 2


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(o=None), I), (dict(table=None), I), (dict(T=-1), I),
    (dict(n=-1), I), (dict(H=0), I), (dict(H_kv=0), I), (dict(H_kv=3), I), (dict(D=0), I), (dict(D=96), U), (dict(D=256), U),
    (dict(dtype=2), I), (dict(scale=float("nan")), I), (dict(scale=-0.5), I), (dict(scale=float("inf")), I), (dict(M=-1), I),
    (dict(P=0), I), (dict(P=-16), I), (dict(P=12), U), (dict(P=1), U), (dict(n_pages=-1), I), (dict(n_pages=0), I), (dict(ts=-1), I),
    (dict(P=1 << 20, M=1 << 12), I), (dict(M=0x7fffffff // 16, nb=1 << 60), I), (dict(cu=None), I), (dict(ts=1 << 60), I),
    (dict(q=off(A[0], 8)), I), (dict(k=off(A[1], 8)), I), (dict(cu=off(A[6], 2)), I), (dict(lse=off(A[9], 1)), I),
    (dict(table=off(A[5], 2)), I), (dict(cl=off(A[7], 3)), I), (dict(o=A[0]), I), (dict(o=off(A[1], 256)), I), (dict(lse=A[2]), I),
    (dict(lse=A[5]), I),
    (dict(st=_st(512, 128, 516, 128, *PAGES)), I),                      # out rows 8 bytes off
    (dict(st=_st(512, 120, 512, 128, *PAGES)), I),                      # q's heads overlap
    (dict(st=_st(512, 128, 0, 128, *PAGES)), I),                        # every token of out in one row
    (dict(st=_st(512, 128, 512, 128, 4096, 2048, 132, 4096, 2048, 128)), I),   # rows of kpages 8 bytes off
    (dict(st=_st(512, 128, 512, 128, -4096, 2048, 128, 4096, 2048, 128)), I),
    (dict(st=_st(512, 128, 512, 128, *PAGES[:3], 1 << 60, 2048, 128)), I),
    (dict(ws=None), I), (dict(nb=16), I), (dict(ws=off(A[8], 8)), I), (dict(ws=A[3]), I), (dict(ws=A[1]), I), (dict(ws=A[5]), I),
    (dict(ws=A[6]), I), (dict(ws=A[7]), I), (dict(T=1 << 28, H=16, nb=1 << 60, k=ctypes.c_void_p(1 << 60), v=ctypes.c_void_p(3 << 59),
                                              o=ctypes.c_void_p(1 << 61)), I),
    (dict(dtype=F32, M=1 << 27, nb=1 << 60), I), (dict(P=24, M=0x7fffffff // 24, nb=1 << 60), I),
])
def test_paged_rejects_bad_arguments(attn_lib, kw, code):
    assert paged(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_empty_paged_calls_are_no_ops(attn_lib):
    assert paged(attn_lib, T=0) == OK and paged(attn_lib, n=0) == OK and paged(attn_lib, T=0, n_pages=0) == OK
    assert attn.attn_last_error() == ""


def test_paged_workspace(attn_lib):
    w = attn_lib.attn_fwd_paged_workspace
    assert w(0, 5, 4, 2, 128, 100, 16, 0, BF) == 0 and w(64, 0, 4, 2, 128, 100, 16, 1, BF) == 0
    assert w(1, 1, 32, 8, 128, 100, 16, 0, BF) == 0            # few units: clusters
    assert w(64, 64, 32, 8, 128, 512, 16, 0, BF) > 0
    assert w(64, 64, 32, 8, 128, 512, 16, 0, BF) < w(64, 64, 32, 8, 128, 512, 16, 1, BF)   # rows of one tile, of two
    assert w(8, 8, 4, 2, 64, 64, 16, 0, F32) == 0 and w(1, 1, 4, 2, 64, 64, 16, 0, F32) == 0 and w(1, 1, 4, 2, 64, 6400, 16, 0, F32) > 0
    for bad in ((-1, 1, 4, 2, 64, 9, 16, 0, BF), (4, 3, 4, 2, 64, 9, 16, 0, BF), (4, 1, 4, 3, 64, 9, 16, 0, BF), (4, 1, 4, 2, 64, -1, 16, 0, BF),
                (4, 1, 4, 2, 64, 9, 16, 0, 7)):
        assert w(*bad) == I
    assert w(4, 1, 4, 2, 96, 9, 16, 0, BF) == U and w(4, 1, 4, 2, 64, 9, 17, 0, BF) == U


FREQS = (ctypes.c_double * 64)(*([0.5] * 64))


def append(lib, q=A[0], k=A[1], v=A[2], qo=A[3], ko=None, kp=A[4], vp=A[5], T=64, H=4, H_kv=2, D=128, st=None, n_pages=100, P=16,
           table=A[6], M=20, ts=20, cu=A[7], cl=A[8], n=3, pos=None, f=FREQS, rd=128, il=0, ms=1.0, wq=A[9], wk=A[10], eps=1e-6,
           dtype=BF):
    return lib.attn_rope_append_paged(q, k, v, qo, ko, kp, vp, T, H, H_kv, D, st, n_pages, P, table, M, ts, cu, cl, n, pos, f, rd, il,
                                      ms, wq, wk, eps, dtype, None)


ROWS = (512, 128, 256, 128, 256, 128, 512, 128, 256, 128)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(qo=None), I), (dict(kp=None), I), (dict(vp=None), I),
    (dict(table=None), I), (dict(T=-1), I), (dict(n=-1), I), (dict(H=0), I), (dict(H_kv=0), I), (dict(D=0), I), (dict(D=80), U),
    (dict(P=0), I), (dict(M=-1), I), (dict(n_pages=-1), I), (dict(n_pages=0), I), (dict(P=1 << 20, M=1 << 12), I), (dict(ts=-1), I),
    (dict(dtype=3), I), (dict(rd=3), I), (dict(rd=130), I), (dict(rd=-2), I), (dict(f=None), I), (dict(il=2), I),
    (dict(ms=float("inf")), I), (dict(ms=float("nan")), I), (dict(eps=-1e-6), I), (dict(eps=float("nan")), I), (dict(eps=float("inf")), I),
    (dict(f=(ctypes.c_double * 64)(*([float("nan")] * 64))), I), (dict(cu=None), I), (dict(q=off(A[0], 1)), I), (dict(wq=off(A[9], 1)), I),
    (dict(kp=off(A[4], 1)), I), (dict(cu=off(A[7], 2)), I), (dict(table=off(A[6], 1)), I),
    (dict(qo=A[1]), I), (dict(qo=A[4]), I), (dict(ko=A[3]), I), (dict(kp=A[5]), I), (dict(kp=A[2]), I), (dict(wq=A[3]), I), (dict(wk=A[5]), I),
    (dict(st=_st(*ROWS, 4096, 2048, 64, *PAGES[:3])), I),               # rows of kpages overlap
    (dict(st=_st(*ROWS, 2048, 2048, 128, *PAGES[:3])), I),              # pages overlap
    (dict(st=_st(*ROWS, *PAGES), kp=A[4], vp=off(A[4], 2048)), I),      # vpages in kpages' rows
    (dict(st=_st(0, *ROWS[1:], *PAGES)), I),
])
def test_append_rejects_bad_arguments(attn_lib, kw, code):
    assert append(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_empty_appends_are_no_ops(attn_lib):
    assert append(attn_lib, T=0) == OK and append(attn_lib, n=0) == OK


def norm(lib, q=A[0], k=A[1], qo=A[2], ko=A[3], T=10, H=4, H_kv=2, D=64, st=None, pos=A[4], f=FREQS, rd=64, il=0, ms=1.0, wq=A[5], wk=A[6],
         eps=1e-6, dtype=BF):
    return lib.attn_norm_rope(q, k, qo, ko, T, H, H_kv, D, st, pos, f, rd, il, ms, wq, wk, eps, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(qo=None), I), (dict(ko=None), I), (dict(pos=None), I), (dict(T=-1), I), (dict(H_kv=-1), I),
    (dict(D=48), U), (dict(rd=5), I), (dict(eps=-1.0), I), (dict(qo=off(A[0], 128)), I), (dict(qo=A[5]), I), (dict(qo=A[3]), I),
    (dict(pos=off(A[4], 1)), I), (dict(dtype=F32, wk=off(A[6], 2)), I),
])
def test_norm_rejects_bad_arguments(attn_lib, kw, code):
    assert norm(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def step(lib, table=A[0], cl=A[1], n=3, M=5, ts=5, n_pages=50, P=16, par=A[2], new=A[3], pin=A[4], n_out=4, out=A[5], os=5, lo=A[6], c=A[7],
         fr=A[8], ws=A[9], nb=1 << 20):
    return lib.attn_pages_step(table, cl, n, M, ts, n_pages, P, par, new, pin, n_out, out, os, lo, c, fr, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(out=None), dict(lo=None), dict(c=None), dict(fr=None), dict(ws=None), dict(nb=8), dict(ws=off(A[9], 4)),
    dict(n=-1), dict(n_out=-1), dict(M=-1), dict(n_pages=-1), dict(P=0), dict(P=1 << 20, M=1 << 12), dict(par=None), dict(ts=-5),
    dict(os=4), dict(out=A[0]), dict(lo=A[1]), dict(c=A[2]), dict(fr=A[3]), dict(ws=A[4]), dict(lo=A[7]), dict(cl=off(A[1], 2)),
    dict(n_out=1 << 20, M=1 << 10, os=1 << 10, nb=1 << 40), dict(n_pages=1 << 30, nb=1 << 40),
])
def test_step_rejects_bad_arguments(attn_lib, kw):
    assert step(attn_lib, **kw) == I
    assert attn.attn_last_error() != ""


def compact(lib, table=A[0], cl=A[1], n=3, M=5, ts=5, n_pages=50, P=16, pin=A[4], out=A[5], os=5, c=A[7], fr=A[8], ws=A[9], nb=1 << 20):
    return lib.attn_pages_compact(table, cl, n, M, ts, n_pages, P, pin, out, os, c, fr, ws, nb, None)


@pytest.mark.parametrize("kw", [dict(table=None), dict(out=None), dict(c=None), dict(fr=None), dict(ws=None), dict(nb=8), dict(out=A[0]),
                                dict(c=A[4]), dict(P=-1), dict(os=3)])
def test_compact_rejects_bad_arguments(attn_lib, kw):
    assert compact(attn_lib, **kw) == I
    assert attn.attn_last_error() != ""


def copy(lib, k=A[0], v=A[1], layers=2, n_pages=50, H_kv=2, P=16, D=64, st=None, c=A[2], n=7, dtype=BF):
    return lib.attn_pages_copy(k, v, layers, n_pages, H_kv, P, D, st, c, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), I), (dict(v=None), I), (dict(c=None), I), (dict(layers=-1), I), (dict(n_pages=-1), I), (dict(H_kv=0), I), (dict(P=0), I),
    (dict(D=0), I), (dict(D=32), U), (dict(n=-1), I), (dict(dtype=4), I), (dict(k=off(A[0], 1)), I), (dict(c=off(A[2], 2)), I), (dict(v=A[0]), I),
    (dict(c=A[1]), I), (dict(st=_st(1, 2048, 1024, 64, 1 << 17, 2048, 1024, 64)), I), (dict(st=_st(1 << 60, 2048, 1024, 64) ), I),
    (dict(H_kv=1 << 16, P=1 << 16), I),
])
def test_copy_rejects_bad_arguments(attn_lib, kw, code):
    if kw.get("st") is not None and len(kw["st"]) == 4:
        kw = dict(st=_st(*list(kw["st"]), 1 << 17, 2048, 1024, 64))
    assert copy(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_empty_copies_are_no_ops(attn_lib):
    assert copy(attn_lib, layers=0) == OK and copy(attn_lib, n_pages=0) == OK and copy(attn_lib, n=0) == OK


def test_halves_of_one_tensor_are_two_pools(attn_lib):
    """(n_pages, 2, H_kv, P, D): accepted as pools (the call goes on to refuse something else)."""
    st = _st(*ROWS, 2 * 4096, 2048, 128, 2 * 4096, 2048, 128)
    assert append(attn_lib, st=st, kp=A[4], vp=off(A[4], 4096 * 2), wq=A[3]) == I and "overlaps a weight" in attn.attn_last_error()
    assert append(attn_lib, st=st, kp=A[4], vp=off(A[4], 4096 * 2 - 256)) == I and "kpages overlaps vpages" in attn.attn_last_error()


def test_checked_paths_refuse_cpu_tensors(attn_lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool, t, f = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for call in (lambda: attn.attn_fwd_paged(x, pool, pool, t), lambda: attn.attn_norm_rope(x, None, t[0], f),
                 lambda: attn.attn_rope_append_paged(x, x, x, pool, pool, t, f), lambda: attn.attn_pages_step(t, None, 3, 16),
                 lambda: attn.attn_pages_compact(t, None, 3, 16), lambda: attn.attn_pages_copy(pool, pool, t)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("name,n", [("paged", 10), ("norm_rope", 11), ("append_paged", 17), ("pages_step", 8), ("pages_compact", 6),
                                    ("pages_copy", 3)])
def test_the_binding_leaves_other_calls(attn_lib, name, n):
    f = getattr(attn._native or attn._load_native(), name)
    assert f() is None and f(*[None] * n) is None and f(*["x"] * n) is None and f(*[torch.zeros(2, 2, 64)] * n) is None


def test_bind_paged_refuses_bad_addresses(attn_lib):
    native = attn._native or attn._load_native()
    if isinstance(native, attn._NoBinding):
        pytest.skip("no binding")
    for bad in ((), (1,) * 7, (0,) * 8):
        with pytest.raises((TypeError, ValueError)):
            native.bind_paged(*bad)
