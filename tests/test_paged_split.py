"""The division of paged attention's work (csrc/paged_tc.cu) restated on the host: every
K/V tile of every unit is taken by exactly one CTA, in runs that the merge finds."""
import random

import pytest

KN, UNIT_COST, MIN_TILES, WEIGHT_TWO = 128, 5, 2, 6


def cdiv(a, b):
    return -(-a // b)


class Units:
    """The axis counts quarters of a key; a sequence of more tokens than one row tile holds has units of two."""

    def __init__(self, n, L, tokens, one_tile):
        self.n, self.L, self.tokens = n, L, tokens
        self.nu = cdiv(n, tokens)
        self.step = min(tokens, n)
        self.two = n > one_tile
        self.weight = WEIGHT_TWO if self.two else 4
        self.tile = self.weight * KN
        self.base = self.weight * (max(L - n, 0) + KN - 1) + UNIT_COST * KN * 4

    def at(self, u):
        return u * self.base + u * (u + 1) // 2 * self.step * self.weight

    def keys(self, u):
        return max(0, min(self.L, self.L - self.n + min((u + 1) * self.tokens, self.n)))

    def tiles(self, u):
        return max(1, cdiv(self.keys(u), KN))

    def cut(self, x, nt):
        if x >= nt * self.tile:
            return nt
        return 0 if x <= 0 else cdiv(x, self.tile)


def runs_of(seqs, per, tokens, one_tile, grid, cta):
    """The (sequence, head, unit, first tile, tiles) of one CTA, walked as its loading warp does."""
    cost = [Units(n, L, tokens, one_tile).at(cdiv(n, tokens)) * per if n else 0 for n, L in seqs]
    total = sum(cost)
    N = max(1, min(total // (4 * KN * MIN_TILES), grid))
    if cta >= N or total == 0:
        return [], None, N, total
    lo, hi = total * cta // N, total * (cta + 1) // N
    b, base = 0, 0
    while base + cost[b] <= lo:
        base += cost[b]
        b += 1
    units = Units(*seqs[b], tokens, one_tile)
    one = units.at(units.nu)
    hs, pos = divmod(lo - base, one)
    pos = base + hs * one
    u, top = 0, units.nu
    while top - u > 1:
        mid = (u + top) // 2
        if units.at(mid) <= lo - pos:
            u = mid
        else:
            top = mid
    pos += units.at(u)
    state = [b, hs, u, 0, pos, units]

    def advance():
        b, hs, u, _, pos, units = state
        pos += units.at(u + 1) - units.at(u)
        u += 1
        if u == units.nu:
            u, hs = 0, hs + 1
            if hs == per:
                hs, b = 0, b + 1
                while b < len(seqs) and seqs[b][0] == 0:
                    b += 1
                if b < len(seqs):
                    units = Units(*seqs[b], tokens, one_tile)
        state[:] = [b, hs, u, 0, pos, units]

    state[3] = units.cut(lo - pos, units.tiles(u))
    if state[3] == units.tiles(u):
        advance()
    runs, rec = [], None
    while state[0] < len(seqs) and state[4] < hi:
        b, hs, u, j, pos, units = state
        nt = units.tiles(u)
        n = units.cut(hi - pos, nt) - j
        if n <= 0:
            break
        runs.append((b, hs, u, j, n))
        if j == 0 and n < nt:
            assert rec is None
            rec = (b, hs, u, ((pos + (nt - 1) * units.tile + 1) * N - 1) // total)
        if j + n == nt:
            advance()
        else:
            state[3] = j + n
            break  # hi is reached
    return runs, rec, N, total


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_every_part_found(seed):
    r = random.Random(seed)
    one_tile = r.choice((1, 2, 16, 25, 32, 64, 128))
    tokens = one_tile * r.choice((1, 2))
    per = r.choice((1, 2, 8))
    seqs = []
    for _ in range(r.choice((1, 2, 5, 40))):
        n = r.choice((0, 1, 1, 1, tokens, tokens + 1, r.randint(1, 700)))
        L = r.choice((0, n // 2, n, n + 1, n + r.randint(0, 3000), n + 127))
        seqs.append((n, L))
    grid = r.choice((1, 3, 152))
    taken, recs, parts = set(), {}, {}
    for cta in range(grid):
        runs, rec, N, _ = runs_of(seqs, per, tokens, one_tile, grid, cta)
        for b, hs, u, j, n in runs:
            for t in range(j, j + n):
                assert (b, hs, u, t) not in taken
                taken.add((b, hs, u, t))
            whole = n == Units(*seqs[b], tokens, one_tile).tiles(u)
            if not whole:
                # slot 2 cta + 1 for the beginning, 2 cta for what goes on: one each a CTA
                assert parts.setdefault((cta, j == 0), (b, hs, u)) == (b, hs, u)
        if rec:
            recs[cta] = rec
    want = {(b, hs, u, t) for b, (n, L) in enumerate(seqs) if n for hs in range(per)
            for u in range(cdiv(n, tokens)) for t in range(Units(n, L, tokens, one_tile).tiles(u))}
    assert taken == want
    cut = {v for v in parts.values()}
    assert {rec[:3] for rec in recs.values()} == cut
    for cta, (b, hs, u, last) in recs.items():
        assert parts[(cta, True)] == (b, hs, u) and last > cta
        for c in range(cta + 1, last + 1):
            assert parts[(c, False)] == (b, hs, u)
        assert all(parts.get((c, False)) != (b, hs, u) for c in range(last + 1, grid))


def test_axis_holds_every_unit():
    """A unit's share holds its tiles, and the host's bound on the axis holds all of them."""
    r = random.Random(5)
    for _ in range(3000):
        one_tile = r.choice((1, 16, 25, 64, 128))
        tokens = 2 * one_tile
        n, L = r.randint(1, 2000), r.randint(0, 5000)
        u = Units(n, L, tokens, one_tile)
        for i in range(u.nu):
            assert u.tiles(i) * u.tile <= u.at(i + 1) - u.at(i)
        assert u.at(u.nu) <= (1 + n / one_tile) * (WEIGHT_TWO * (L + n + KN) + 4 * KN * UNIT_COST)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 16, 33, 64, 100, 128, 129, 200, 300])
def test_rows_of_a_tile_hold_every_head_once(G):
    """Groups of heads, heads and tokens of a tile as the host sets them."""
    groups = cdiv(G, 128)
    heads = cdiv(G, groups)
    tokens = 128 // heads
    assert 1 <= heads <= 128 and tokens >= 1
    seen = [g * heads + h for g in range(groups) for h in range(heads) if g * heads + h < G]
    assert seen == list(range(G))
