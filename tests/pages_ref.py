"""The table of pages by its definition, one entry after the other (test helper)."""
from __future__ import annotations


def step(table, lens, n_pages, P, parents=None, new_len=None, pinned=None):
    """(table, lengths, copies, free) of attn_pages_step."""
    M = len(table[0]) if table else 0
    most = M * P
    lens = [min(max(L, 0), most) for L in lens]
    if parents is None:
        parents = list(range(len(table)))
    some = [0 <= p < len(table) for p in parents]
    L = [lens[p] if ok else 0 for p, ok in zip(parents, some)]
    new = list(L) if new_len is None else [min(max(n, 0), most) for n in new_len]
    keep = [min(a, b) for a, b in zip(L, new)]
    old = [table[p] if ok else [-1] * M for p, ok in zip(parents, some)]

    def page(p):
        return 0 <= p < n_pages

    full = {p for b, row in enumerate(old) for p in row[:keep[b] // P] if page(p)}
    full |= {p for p in range(n_pages) if pinned and pinned[p]}
    held, stays = set(full), []
    for b, row in enumerate(old):
        last = row[keep[b] // P] if keep[b] % P else -1
        ok = page(last) and last not in held
        stays.append(ok)
        if ok:
            held.add(last)
    free = [p for p in range(n_pages) if p not in held]
    out, copies, given = [], [], 0
    for b, row in enumerate(old):
        n_full, part = divmod(keep[b], P)
        kept = n_full + stays[b]
        o = [-1] * M
        for i in range(-(-new[b] // P)):
            if i < kept and page(row[i]):
                o[i] = row[i]
            else:
                o[i] = free[given] if given < len(free) else -1
                given += 1
        out.append(o)
        c = part and not stays[b] and page(row[n_full]) and o[n_full] >= 0
        copies.append([row[n_full], o[n_full], part] if c else [-1, -1, 0])
    return out, new, copies, len(free) - given


def compact(table, lens, n_pages, P, pinned=None):
    """(table, copies, free) of attn_pages_compact."""
    M = len(table[0]) if table else 0
    rows = [[p for p in row[:-(-min(max(L, 0), M * P) // P)]] for row, L in zip(table, lens)]
    held = {p for row in rows for p in row if 0 <= p < n_pages}
    pins = {p for p in range(n_pages) if pinned and pinned[p]}
    n = len(held | pins)
    holes = [p for p in range(n) if p not in held and p not in pins]
    moved = sorted(p for p in held if p >= n and p not in pins)
    to = dict(zip(moved, holes))
    out = [[to.get(p, p) if 0 <= p < n_pages else -1 for p in row] + [-1] * (M - len(row)) for row in rows]
    copies = [[p, to[p], P] for p in moved]
    return out, copies + [[-1, -1, 0]] * ((n_pages + 1) // 2 - len(copies)), n_pages - n
