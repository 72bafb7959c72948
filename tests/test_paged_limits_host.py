"""Sizes and overlaps that the calls of a paged cache refuse on the host, before any CUDA
call: what their kernels count in 32 bits, and what they write over what they read.  The
addresses are never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

import transformer_scaled_dot_fwd_gb300 as attn
from test_paged_host import A, I, compact, copy, step

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
