"""Sizes and overlaps that the calls of a paged cache refuse on the host, before any CUDA
call: what their kernels count in 32 bits, and what they write over what they read.  The
addresses are never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

import transformer_scaled_dot_fwd_gb300 as attn
from test_paged_host import A, BF, F32, I, append, compact, copy, norm, off, paged, step

MOST = 1 << 29  # rows of a new table, pairs of a list: three entries of each are counted in 32 bits


@pytest.mark.parametrize("M", [0, 1])
@pytest.mark.parametrize("n", [MOST + 1, 715827883, 0x7fffffff])
def test_tables_of_too_many_rows_are_refused(attn_lib, n, M):
    """With few entries a row the entries alone do not bound the rows."""
    far = [ctypes.c_void_p(1 << 40 | i << 36) for i in range(4)]
    kw = dict(n_out=n, M=M, ts=M, os=M, new=None, par=far[0], out=far[1], lo=far[2], c=far[3], ws=ctypes.c_void_p(1 << 50), nb=1 << 40)
    assert step(attn_lib, **kw) == I and "too large" in attn.attn_last_error()
    kw = dict(n=n, M=M, ts=M, os=M, cl=None, pin=None, table=far[0], out=far[1], c=far[2], ws=ctypes.c_void_p(1 << 50), nb=1 << 40)
    assert compact(attn_lib, **kw) == I and "too large" in attn.attn_last_error()


@pytest.mark.parametrize("n", [MOST + 1, 1431655766, 0x7fffffff])
def test_lists_of_too_many_copies_are_refused(attn_lib, n):
    assert copy(attn_lib, n=n) == I and "too large" in attn.attn_last_error()


def test_the_largest_compaction_has_a_list_that_can_be_copied(attn_lib):
    """A pool of 2^30 - 1 pages, the most that attn_pages_compact takes, fills a list of 2^29 pairs."""
    assert ((1 << 30) - 1 + 1) // 2 == MOST
    # accepted as far as its size goes: the next check refuses what it overlaps
    assert copy(attn_lib, n=MOST, c=A[0]) == I and "copies overlaps kpages" in attn.attn_last_error()


# the arrays that say where a call's rows lie: T 100, n_seq 3, a table of 3 x 20 entries
INDEX = {"page_table": (A[5], 3 * 20 * 4), "cu_seqlens": (A[6], 4 * 4), "cache_len": (A[7], 3 * 4)}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", ["o", "lse"])
@pytest.mark.parametrize("name", INDEX)
def test_attention_refuses_outputs_over_its_index_arrays(attn_lib, name, out, dtype):
    """Other blocks, and the merge that follows, still read them."""
    p, n = INDEX[name]
    size = 100 * 4 * (128 * (2 if dtype == BF else 4) if out == "o" else 4)
    arg = {"page_table": "table", "cu_seqlens": "cu", "cache_len": "cl"}[name]
    base = off(p, 1 << 20)
    for at in (0, size - 4):  # the array's first bytes, its last ones at the output's front
        assert paged(attn_lib, dtype=dtype, **{out: base, arg: off(base, at)}) == I
        assert attn.attn_last_error().endswith(f"overlaps {name}"), attn.attn_last_error()
    assert paged(attn_lib, dtype=dtype, **{out: off(base, (n - 1) // 16 * 16), arg: base}) == I
    assert attn.attn_last_error().endswith(f"overlaps {name}")
    # side by side: the call goes on to refuse something else
    assert paged(attn_lib, ws=None, **{out: base, arg: off(base, 100 * 4 * 128 * 2)}) == I and "workspace" in attn.attn_last_error()


APPEND_INDEX = {"page_table": ("table", 3 * 20 * 4), "cu_seqlens": ("cu", 16), "cache_len": ("cl", 12), "positions": ("pos", 64 * 4)}


@pytest.mark.parametrize("out", ["qo", "ko", "kp", "vp"])
@pytest.mark.parametrize("name", APPEND_INDEX)
def test_appends_refuse_outputs_over_their_index_arrays(attn_lib, name, out):
    arg, n = APPEND_INDEX[name]
    size = {"qo": 64 * 4 * 128, "ko": 64 * 2 * 128, "kp": 100 * 2 * 16 * 128, "vp": 100 * 2 * 16 * 128}[out] * 2
    base = off(A[12], 1 << 20)
    for at in (0, 256, size - 4):
        assert append(attn_lib, **{out: base, arg: off(base, at)}) == I
        assert attn.attn_last_error().endswith(f"overlaps {name}"), attn.attn_last_error()
    assert append(attn_lib, **{out: off(base, n - 4), arg: base}) == I and attn.attn_last_error().endswith(f"overlaps {name}")


@pytest.mark.parametrize("out", ["qo", "ko"])
def test_norm_refuses_outputs_over_its_positions(attn_lib, out):
    base = off(A[12], 1 << 20)
    assert norm(attn_lib, **{out: base, "pos": off(base, 64)}) == I and attn.attn_last_error().endswith("overlaps positions")
