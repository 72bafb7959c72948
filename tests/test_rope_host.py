"""Host-side tests of the rotary entry points: refusals before any CUDA call
(the fake addresses are never dereferenced), and the frequency helper."""
from __future__ import annotations

import ctypes
import math
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn

Q, K, V, QO, KO, KC, VC, POS = (ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(8))
FREQS = (ctypes.c_double * 64)(*[1.0] * 64)
I, U = attn.ATTN_EINVAL, attn.ATTN_EUNSUPPORTED


def _st(*v):
    return (ctypes.c_longlong * len(v))(*v)


def rope(lib, q=Q, k=K, qo=QO, ko=KO, T=16, H=4, H_kv=2, D=128, st=None, pos=POS, freqs=FREQS, rd=128, inter=0, inv=0,
         ms=1.0, dtype=attn.ATTN_BF16):
    return lib.attn_rope(q, k, qo, ko, T, H, H_kv, D, st, pos, freqs, rd, inter, inv, ms, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(qo=None), I), (dict(ko=None), I), (dict(pos=None), I),
    (dict(freqs=None), I), (dict(T=-1), I), (dict(H=0), I), (dict(H_kv=-1), I), (dict(D=0), I), (dict(D=96), U),
    (dict(D=256), U), (dict(rd=127), I), (dict(rd=130), I), (dict(rd=-2), I), (dict(inter=2), I), (dict(inv=-1), I),
    (dict(ms=float("nan")), I), (dict(ms=float("inf")), I), (dict(dtype=5), I),
    (dict(freqs=(ctypes.c_double * 64)(*[math.inf] * 64)), I),
    (dict(q=ctypes.c_void_p(0x100000001)), I), (dict(pos=ctypes.c_void_p(0x800000002)), I),
    (dict(qo=K), I),                                                     # q_out overlaps k
    (dict(ko=Q), I),                                                     # k_out overlaps q
    (dict(qo=ctypes.c_void_p(Q.value + 256)), I),                        # shifted by one head: not in place
    (dict(qo=Q, st=_st(512, 128, 256, 128, 1024, 128, 256, 128)), I),    # same address, other strides
    (dict(st=_st(512, 64, 256, 128, 512, 128, 256, 128)), I),            # heads of q overlap
    (dict(st=_st(512, 128, 256, 128, 0, 128, 256, 128)), I),             # every token writes one row
    (dict(st=_st(512, 128, 256, 128, -512, 128, 256, 128)), I),
    # q_out as the columns just before k's in one matrix, but one head too wide
    (dict(qo=ctypes.c_void_p(K.value - 3 * 256), st=_st(512, 128, 1024, 128, 1024, 128, 256, 128)), I),
])
def test_rope_rejects_bad_arguments(attn_lib, kw, code):
    assert rope(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def append(lib, q=Q, k=K, v=V, qo=QO, ko=None, kc=KC, vc=VC, T=16, H=4, H_kv=2, D=128, st=None, B=2, Skv=64, cu=POS,
           cl=POS, pos=POS, freqs=FREQS, rd=64, inter=0, ms=1.0, dtype=attn.ATTN_F32):
    return lib.attn_rope_append(q, k, v, qo, ko, kc, vc, T, H, H_kv, D, st, B, Skv, cu, cl, pos, freqs, rd, inter, ms,
                                dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), I), (dict(k=None), I), (dict(v=None), I), (dict(qo=None), I), (dict(kc=None), I), (dict(vc=None), I),
    (dict(B=0), I), (dict(Skv=-1), I), (dict(H_kv=0), I), (dict(D=80), U),
    (dict(cu=None, T=15), I),                                            # no cu_seqlens: T / B tokens each
    (dict(vc=KC), I), (dict(kc=Q), I), (dict(qo=VC), I), (dict(qo=V), I), (dict(ko=V), I), (dict(ko=QO), I),
    (dict(kc=ctypes.c_void_p(KC.value + 8)), I), (dict(cl=ctypes.c_void_p(0x800000001)), I),
])
def test_append_rejects_bad_arguments(attn_lib, kw, code):
    assert append(attn_lib, **kw) == code
    assert attn.attn_last_error() != ""


def test_no_tokens_is_a_no_op(attn_lib):
    assert rope(attn_lib, T=0) == attn.ATTN_OK
    assert append(attn_lib, T=0) == attn.ATTN_OK
    assert attn.attn_last_error() == ""


def test_binding_refusals(attn_lib):
    x = torch.zeros(4, 2, 64)
    f = attn.attn_rope_frequencies(64)
    with pytest.raises(ValueError):
        attn.attn_rope(x, None, torch.zeros(4, dtype=torch.int32), f)  # CPU tensors
    for bad in (f.float(), f[::2], f.reshape(2, -1), [1.0] * 32, attn.attn_rope_frequencies(66)):
        with pytest.raises(ValueError):
            attn._freqs_arg(bad, 64)


def test_frequencies():
    w = attn.attn_rope_frequencies(8, theta=10000.0)
    assert w.dtype == torch.float64 and w.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    lin = attn.attn_rope_frequencies(8, scaling="linear", factor=4.0)
    assert lin.tolist() == pytest.approx([x / 4 for x in w.tolist()], rel=1e-14)
    ntk = attn.attn_rope_frequencies(8, scaling="ntk", factor=4.0)
    # the highest frequency stays, the lowest is divided by the factor
    assert ntk[0] == w[0] and float(ntk[-1]) == pytest.approx(float(w[-1]) / 4, rel=1e-12)
    L = 2 * math.pi * 100  # turns over the original context: 100, 10, 1, 0.1
    wl = attn.attn_rope_frequencies(8, scaling="wavelength", factor=4.0, original_len=L, low=1.0, high=20.0)
    s = (10 - 1) / 19
    assert wl.tolist() == pytest.approx([1.0, 0.1 * ((1 - s) / 4 + s), 0.01 / 4, 0.001 / 4], rel=1e-12)
    assert attn.attn_rope_frequencies(0).numel() == 0
    assert attn.attn_rope_frequencies(2, scaling="ntk", factor=4.0).tolist() == [1.0]
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, scaling="cubic"), dict(rotary_dim=8, theta=0.0),
                dict(rotary_dim=8, scaling="wavelength", low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            attn.attn_rope_frequencies(**bad)


def _pi(digits=120):
    """pi as a Fraction, by Machin's formula in integers."""
    one = 10 ** (digits + 10)

    def arctan_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term, k = term // (n * n), k + 1
        return total

    return Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


def test_turns_are_right_to_the_last_unit(tmp_path):
    """Frequencies as 64-bit fractions of a turn (csrc/rope_turns.h, compiled here for
    the CPU) against exact arithmetic: within one unit, both signs."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    csrc = os.path.join(os.path.dirname(os.path.abspath(attn.__file__)), "csrc")
    (tmp_path / "t.cpp").write_text('#include "rope_turns.h"\n'
                                    'extern "C" unsigned long long turns(double w) { return attn::rope_turns(w); }\n')
    subprocess.run([gxx, "-O2", "-shared", "-fPIC", "-I", csrc, str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t.so")],
                   check=True)
    turns = ctypes.CDLL(str(tmp_path / "t.so")).turns
    turns.argtypes, turns.restype = [ctypes.c_double], ctypes.c_ulonglong
    two_pi = 2 * _pi()
    r = random.Random(7)
    ws = [0.0, -0.0, 1.0, 2 * math.pi, math.pi, 1e-320, 6.283185307179587, float(2 ** 40 - 1), 1.5e-9]
    ws += [10000.0 ** (-p / 32) for p in range(32)] + [r.uniform(-1, 1) * 2.0 ** r.randint(-70, 40) for _ in range(2000)]
    for w in ws:
        for x in (w, -w):
            off = (turns(x) - Fraction(x) / two_pi * 2 ** 64) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= 1, x


def test_a_cache_of_no_rows_needs_no_memory(attn_lib):
    """NULL caches pass the check when Skv = 0 (and the call then fails on the overlap,
    before any CUDA call), not otherwise."""
    assert append(attn_lib, kc=None, vc=None, Skv=0, qo=V) == I and "overlaps" in attn.attn_last_error()
    for kw in (dict(kc=None, vc=None), dict(kc=None), dict(vc=None), dict(kc=None, vc=None, Skv=1)):
        assert append(attn_lib, qo=V, **kw) == I and "NULL" in attn.attn_last_error()
    assert append(attn_lib, kc=None, vc=None, Skv=0, T=0) == attn.ATTN_OK
