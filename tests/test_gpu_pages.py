"""GPU tests of the table of pages (attn_pages_step, attn_pages_compact) against its
definition, entry by entry, and of attn_pages_copy.  Everything is a whole number or a copy:
equal, not close."""
from __future__ import annotations

import random

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
import pages_ref as ref

pytestmark = pytest.mark.gpu


def ints(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


def state(r, B, M, P, n_pages, share=0.5, bad=0.1):
    """Rows over a pool, some of them sharing the front of another, with a few entries that are no pages."""
    ids = list(range(n_pages))
    r.shuffle(ids)
    table, lens = [], []
    for b in range(B):
        L = r.choice((0, 1, P, M * P, r.randint(0, M * P), r.randint(0, M * P)))
        n = -(-L // P)
        row, front = [], 0
        if b and r.random() < share:
            other = r.randrange(b)
            front = min(n, -(-lens[other] // P), r.randint(0, M))
            row = table[other][:front]
        row += [ids.pop() if ids else -1 for _ in range(n - front)]
        row = [r.choice((-1, n_pages, -7, 2 ** 31 - 1)) if r.random() < bad else p for p in row]
        table.append(row + [r.randint(-3, n_pages + 3) for _ in range(M - n)])
        lens.append(L)
    return table, lens


def run_step(table, lens, n_pages, P, M, parents, new_len, pinned, **kw):
    B = len(table)
    return attn.attn_pages_step(ints(table, (B, M)), ints(lens), n_pages, P,
                                parents=None if parents is None else ints(parents),
                                new_len=None if new_len is None else ints(new_len),
                                pinned=None if pinned is None else ints(pinned), **kw)


def compare(got, want):
    for g, w in zip(got, want):
        assert g.dtype == torch.int32
        assert g.flatten().tolist() == ints(w).flatten().tolist()


@pytest.mark.parametrize("seed", range(40))
@pytest.mark.parametrize("spare", [0, 262200])
def test_step(gpu, seed, spare):
    """spare: free pages behind those that matter, for a pool that takes a launch a step."""
    r = random.Random(seed)
    B, M, P = r.choice((1, 2, 9, 40)), r.choice((1, 2, 5, 31, 33, 70)), r.choice((1, 8, 16, 37))
    n_pages = r.choice((1, 31, 32, 33, 100, B * M, 2 * B * M + 5))
    table, lens = state(r, B, M, P, n_pages, bad=r.choice((0.0, 0.1)))
    n_out = r.choice((B, B, 1, 2 * B + 3))
    parents = None if n_out == B and r.random() < 0.4 else [r.choice((r.randrange(B), r.randrange(B), 0, -1, B)) for _ in range(n_out)]
    new_len = None if r.random() < 0.2 else [r.choice((0, r.randint(0, M * P), M * P, M * P + 9, -4)) for _ in range(n_out)]
    if new_len is not None and r.random() < 0.5:  # mostly a step of one token
        base = [lens[p] if 0 <= p < B else 0 for p in (parents or range(B))]
        new_len = [L + 1 for L in base]
    pinned = None if r.random() < 0.5 else [int(r.random() < 0.1) * r.choice((1, -1, 5)) for _ in range(n_pages)]
    if spare:  # entries that were no pages may be now
        pinned = pinned and pinned + [0] * spare
        n_pages += spare
    got = run_step(table, lens, n_pages, P, M, parents, new_len, pinned)
    compare(got, ref.step(table, lens, n_pages, P, parents, new_len, pinned))


@pytest.mark.parametrize("seed", range(20))
@pytest.mark.parametrize("spare", [0, 262200])
def test_compact(gpu, seed, spare):
    r = random.Random(100 + seed)
    B, M, P = r.choice((1, 2, 9, 40)), r.choice((1, 2, 5, 33)), r.choice((1, 8, 16))
    n_pages = r.choice((1, 31, 32, 33, 100, 3 * B * M))
    table, lens = state(r, B, M, P, n_pages)
    pinned = None if r.random() < 0.5 else [int(r.random() < 0.2) for _ in range(n_pages)]
    if spare:
        table = [[p + spare // 2 if p < n_pages and r.random() < 0.3 else p for p in row] for row in table]
        pinned = pinned and pinned + [0] * spare
        n_pages += spare
    got = attn.attn_pages_compact(ints(table, (B, M)), ints(lens), n_pages, P, pinned=None if pinned is None else ints(pinned))
    compare(got, ref.compact(table, lens, n_pages, P, pinned))


@pytest.mark.parametrize("n_pages,B", [(100003, 1500), (262144, 2048), (262145, 300), (90000, 2049)])
def test_a_large_pool(gpu, n_pages, B):
    """More words of bits and more rows than a block has threads; the largest of the one-launch form and beyond."""
    r = random.Random(7)
    M, P = 40, 16
    table, lens = state(r, B, M, P, n_pages, share=0.2, bad=0.0)
    parents = [r.randrange(B) for _ in range(B)]
    new_len = [min(M * P, lens[p] + r.randint(0, 40)) for p in parents]
    compare(run_step(table, lens, n_pages, P, M, parents, new_len, None), ref.step(table, lens, n_pages, P, parents, new_len))
    got = attn.attn_pages_compact(ints(table, (B, M)), ints(lens), n_pages, P)
    compare(got, ref.compact(table, lens, n_pages, P))


def test_beams_fork_and_sequences_end_and_begin(gpu):
    """Three beams go on from one, its partly filled page stays with the first; a page of an
    ended sequence is given out in the same call; an empty row begins."""
    P, M, n_pages = 4, 4, 8
    table = [[5, 2, -1, -1], [7, 0, 3, -1], [-1] * 4]
    lens = [6, 9, 0]
    got = run_step(table, lens, n_pages, P, M, [1, 1, 1, -1], [10, 10, 10, 3], None)
    # kept: 7 and 0 full, 3 by the first row; free: 1, 2, 4, 5, 6
    assert got[0].tolist() == [[7, 0, 3, -1], [7, 0, 1, -1], [7, 0, 2, -1], [4, -1, -1, -1]]
    assert got[1].tolist() == [10, 10, 10, 3]
    assert got[2].tolist() == [[-1, -1, 0], [3, 1, 1], [3, 2, 1], [-1, -1, 0]]
    assert got[3].item() == 2


def test_cut_into_a_shared_page(gpu):
    """A sequence cut back into a page that another holds full copies it before it appends."""
    got = run_step([[4, 1], [4, 2]], [8, 5], 6, 4, 2, None, [3, 6], None)
    assert got[0].tolist() == [[0, -1], [4, 2]] and got[2].tolist() == [[4, 0, 3], [-1, -1, 0]]
    # the same, the page pinned and not shared
    got = run_step([[4, 1]], [8], 6, 4, 2, None, [3], [0, 0, 0, 0, 1, 0])
    assert got[0].tolist() == [[0, -1]] and got[2].tolist() == [[4, 0, 3]]


def test_a_shortage_is_told_and_mended(gpu):
    P, M, n_pages = 8, 4, 3
    first = run_step([[0, -1, -1, -1], [1, -1, -1, -1]], [8, 8], n_pages, P, M, None, [24, 20], None)
    assert first[0].tolist() == [[0, 2, -1, -1], [1, -1, -1, -1]] and first[3].item() == -3
    again = attn.attn_pages_step(first[0], first[1], n_pages, P, parents=ints([0]))
    assert again[0].tolist() == [[0, 2, 1, -1]] and again[3].item() == 0


def test_given_outputs_empty_tables_and_streams(gpu):
    r = random.Random(5)
    table, lens = state(r, 6, 5, 16, 60)
    want = run_step(table, lens, 60, 16, 5, None, None, None)
    out = [torch.empty_like(t) for t in want]
    got = run_step(table, lens, 60, 16, 5, None, None, None, out=out)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(want, out))
    wide = torch.full((6, 9), 3, dtype=torch.int32, device="cuda")
    wide[:, :5] = ints(table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.attn_pages_step(wide[:, :5], ints(lens), 60, 16, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    none = attn.attn_pages_step(torch.empty(0, 5, dtype=torch.int32, device="cuda"), None, 7, 16)
    assert none[0].shape == (0, 5) and none[3].item() == 7
    full = attn.attn_pages_step(ints([[1, 0]]), None, 4, 16, new_len=ints([40]))
    assert full[0].tolist() == [[1, 0]] and full[1].tolist() == [32]
    moved = attn.attn_pages_compact(ints([[6, 0]]), None, 7, 16)
    assert moved[0].tolist() == [[1, 0]] and moved[1][0].tolist() == [6, 1, 16]
    no_pages = attn.attn_pages_step(ints([[1, 0]]), ints([0]), 0, 16, new_len=ints([3]))
    assert no_pages[0].tolist() == [[-1, -1]] and no_pages[3].item() == -1


def test_captured(gpu):
    r = random.Random(6)
    table, lens = state(r, 12, 9, 16, 150)
    t, L, par, new = ints(table), ints(lens), ints(list(range(12))), ints(lens)
    attn.attn_pages_step(t, L, 150, 16, parents=par, new_len=new)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = attn.attn_pages_step(t, L, 150, 16, parents=par, new_len=new)
        moved = attn.attn_pages_compact(got[0], got[1], 150, 16)
    for seed in (1, 2, 3):
        r = random.Random(seed)
        table, lens = state(r, 12, 9, 16, 150)
        parents, new_len = [r.randrange(12) for _ in range(12)], [r.randint(0, 144) for _ in range(12)]
        t.copy_(ints(table)), L.copy_(ints(lens)), par.copy_(ints(parents)), new.copy_(ints(new_len))
        g.replay()
        torch.cuda.synchronize()
        want = ref.step(table, lens, 150, 16, parents, new_len)
        compare(got, want)
        compare(moved, ref.compact(want[0], want[1], 150, 16))


# ------------------------------------------------------------ copies

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers,H_kv,P,D,layout", [(0, 2, 16, 128, "heads"), (3, 1, 5, 64, "heads"), (2, 8, 64, 128, "rows"),
                                                    (1, 3, 16, 64, "halves"), (0, 2, 8, 64, "odd")])
def test_copies(gpu, dtype, layers, H_kv, P, D, layout):
    r = random.Random(layers + P)
    n_pages = 40
    lead = (layers,) if layers else ()
    if layout == "rows":
        k, v = (torch.randn(*lead, n_pages, P, H_kv, D, device="cuda").to(dtype).transpose(-2, -3) for _ in range(2))
    elif layout == "halves":
        kv = torch.randn(*lead, n_pages, 2, H_kv, P, D, device="cuda").to(dtype)
        k, v = kv[..., 0, :, :, :], kv[..., 1, :, :, :]
    elif layout == "odd":  # rows that allow no 16-byte accesses
        k, v = (torch.randn(*lead, n_pages, H_kv, P, D + 1, device="cuda").to(dtype)[..., 1:] for _ in range(2))
    else:
        k, v = (torch.randn(*lead, n_pages, H_kv, P, D, device="cuda").to(dtype) for _ in range(2))
    ids = list(range(n_pages))
    r.shuffle(ids)
    pairs = [(ids[i], ids[20 + i], r.choice((0, 1, P - 1, P, P + 4, -3))) for i in range(15)]
    pairs.append((ids[0], ids[36], P))  # a page copied twice
    pairs += [(-1, ids[37], P), (ids[1], n_pages, P), (ids[2], -1, P), (2 ** 31 - 1, ids[38], P), (-1, -1, 0)]
    want = [x.clone() for x in (k, v)]
    for x, w in zip((k, v), want):
        for src, dst, rows in pairs:
            if 0 <= src < n_pages and 0 <= dst < n_pages:
                rows = min(max(rows, 0), P)
                w[..., dst, :, :rows, :] = x[..., src, :, :rows, :]
    attn.attn_pages_copy(k, v, ints(pairs))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    attn.attn_pages_copy(k, v, torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_copies_past_32_bits(gpu):
    n_pages, H_kv, P, D = (1 << 31) // (8 * 64 * 128) + 9, 8, 64, 128
    k, v = (torch.zeros(n_pages, H_kv, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[n_pages - 2], v[3] = 1.0, 2.0
    attn.attn_pages_copy(k, v, ints([[n_pages - 2, n_pages - 1, P], [3, n_pages - 3, 7]]))
    assert bool((k[n_pages - 1] == 1).all()) and bool((v[n_pages - 3, :, :7] == 2).all())
    assert torch.count_nonzero(v[n_pages - 3, :, 7:]) == 0 and torch.count_nonzero(k[3]) == 0
