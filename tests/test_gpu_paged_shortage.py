"""A table of pages whose pool runs out: what the call says, how a server goes on without
losing a token, and what a later call on the short table gives."""
from __future__ import annotations

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
import pages_ref as ref

pytestmark = pytest.mark.gpu
P, M = 4, 4


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def compare(got, want):
    for g, w in zip(got, want):
        assert g.flatten().tolist() == ints(w).flatten().tolist()


def pools(n_pages):
    g = torch.Generator().manual_seed(3)
    return [torch.randn(n_pages, 1, P, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]


def rows_of(pool, table, n):
    return torch.cat([pool[p, 0] for p in table[:-(-n // P)]])[:n]


@pytest.mark.parametrize("spare", [0, 262200])
def test_the_old_table_still_stands(gpu, spare):
    """Three beams of one sequence whose partly filled page two of them need a copy of, with one page left.
    spare: pinned pages, for a pool that takes a launch a step."""
    table, lens = [[0, 1, -1, -1]], [6]
    pinned = [0, 0, 0] + [1] * spare
    n_pages = 3 + spare
    kp, vp = pools(3)
    before = [rows_of(x, table[0], 6).clone() for x in (kp, vp)]
    t, L, pin = ints(table), ints(lens), ints(pinned)
    short = attn.attn_pages_step(t, L, n_pages, P, parents=ints([0, 0, 0]), new_len=ints([7, 7, 7]), pinned=pin)
    compare(short, ref.step(table, lens, n_pages, P, [0, 0, 0], [7, 7, 7], pinned))
    # the third has no page for its last tokens, and nothing to copy them to
    assert short[3].item() == -1 and short[0][2].tolist() == [0, -1, -1, -1] and short[2][2].tolist() == [-1, -1, 0]
    # again from the old table, with a beam less: nothing was lost
    good = attn.attn_pages_step(t, L, n_pages, P, parents=ints([0, 0]), new_len=ints([7, 7]), pinned=pin)
    assert good[3].item() == 0
    x, y = kp.clone(), vp.clone()
    attn.attn_pages_copy(x, y, good[2])
    for b in range(2):
        for pool, want in zip((x, y), before):
            assert torch.equal(rows_of(pool, good[0][b].tolist(), 6), want)
    # or on from the short table, its copies made, with that beam cut back to the pages it has
    cut = attn.attn_pages_step(short[0], short[1], n_pages, P, parents=ints([0, 1, 2]), new_len=ints([7, 7, 4]), pinned=pin)
    assert cut[3].item() == 0 and cut[0][2].tolist() == [0, -1, -1, -1] and cut[1].tolist() == [7, 7, 4]
    attn.attn_pages_copy(kp, vp, short[2])
    attn.attn_pages_copy(kp, vp, cut[2])
    for b, n in enumerate((6, 6, 4)):
        for pool, want in zip((kp, vp), before):
            assert torch.equal(rows_of(pool, cut[0][b].tolist(), n), want[:n])


@pytest.mark.parametrize("spare", [0, 262200])
def test_a_later_call_gives_pages_without_their_tokens(gpu, spare):
    """The short table's missing entry gets a page when there is one, and no copy: its rows are whatever they were."""
    table, lens, n_pages = [[0, -1, -1, -1], [0, 1, -1, -1]], [7, 7], 3 + spare
    pinned = [0, 0, 0] + [1] * spare
    got = attn.attn_pages_step(ints(table), ints(lens), n_pages, P, new_len=ints([8, 8]), pinned=ints(pinned))
    compare(got, ref.step(table, lens, n_pages, P, None, [8, 8], pinned))
    assert got[0][0].tolist() == [0, 2, -1, -1] and got[2].tolist() == [[-1, -1, 0]] * 2 and got[3].item() == 0
