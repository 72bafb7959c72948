"""Offsets of a paged call that are none (decreasing, so that sequences overlap) make its
axis of keys longer than the host allows for: every sequence may then hold all tokens.  The
kernel takes such an axis for no work before anything is multiplied by it.  Its constants are
read from the source."""
import os
import re

import pytest

import transformer_scaled_dot_fwd_gb300.build as build
from test_paged_split import KN, UNIT_COST, WEIGHT_TWO, Units, cdiv, runs_of

TC = open(os.path.join(build.CSRC, "paged_tc.cu")).read()
API = open(os.path.join(build.CSRC, "api.cu")).read()
MOST_CTAS = 1023


def max_axis():
    m = re.search(r"constexpr long long kMaxAxis = 1ll << (\d+);", TC)
    assert m, "the kernel has no bound on the axis"
    return 1 << int(m.group(1))


def test_what_the_host_lets_through_is_work():
    """The host refuses an axis (of any valid offsets) of more than 4e18 / 1024."""
    assert "if (axis * 1024 > 4e18)" in API and f"if (a.grid > {MOST_CTAS}) a.grid = {MOST_CTAS};" in API
    assert 4e18 / 1024 < max_axis()


def test_products_and_sums_of_the_axis_fit_64_bits():
    most = max_axis()
    assert (most + 1) * MOST_CTAS < 1 << 63          # a place times the number of CTAs
    # a sequence's own part is bounded as the host bounds the whole; a lane stops adding beyond the bound
    assert "total = min(total + t, kMaxAxis + 1);" in TC
    assert 32 * (2 * most + 1) < 1 << 63             # sums over a warp
    assert re.search(r"idle = I >= N \|\| total == 0 \|\| total > kMaxAxis;", TC)


def test_overlapping_sequences_would_pass_them():
    """Offsets 0, T, 0, T, ...: without the bound the products wrap, and the merge would look for parts of CTAs that are
    not there."""
    T, max_len, tokens, per, n_seq = 1 << 20, 1 << 30, 256, 8, 1 << 14
    one = Units(T, max_len, tokens, 128)
    axis = (n_seq + T / 128) * per * (WEIGHT_TWO * (max_len + T + KN) + 4 * KN * UNIT_COST)
    assert axis * 1024 < 4e18                        # the call is accepted
    total = n_seq // 2 * one.at(cdiv(T, tokens)) * per
    assert total > max_axis() and total * 152 > 1 << 63


@pytest.mark.parametrize("cta", [0, 5])
def test_ordinary_overlapping_sequences_are_walked(cta):
    """Below the bound such offsets are work like any other: no CTA leaves its part of the axis."""
    seqs = [(700, 900), (0, 5), (700, 30), (1, 1), (700, 900)]
    runs, rec, N, total = runs_of(seqs, 2, 64, 32, 9, cta)
    assert runs and total < max_axis() and (rec is None or rec[3] < N)
