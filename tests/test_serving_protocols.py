"""CPU models of the mbarrier protocols of the packed prefill and the tree decode
kernels: the prefill and decode protocols (test_barrier_protocols.py) with the
guard warps that pass over the V tiles at the edge of what rows see.

The guard waits for a request that the producer files after issuing a V load,
then for that load, and the MMA warp waits for the guard before it reads the
tile.  Random interleavings must finish, no wait may see its barrier two phases
ahead, a tile must be loaded when the guard passes over it and clean when the
MMA reads it, and an open request's slot must not be filed again.
"""
from __future__ import annotations

import random

import pytest

from test_barrier_protocols import RING, Bar, Hazard, Sched, wait

GUARD_RING = 8
TREE_REQS = 16


def wait_parity(bar, phase):
    """What the hardware tests: the phase in progress has the other parity.  It
    also holds one phase too early, which the guard's request has to rule out."""
    return lambda: (bar.phase - phase) % 2 == 1


def packed_run(items, stages, seed, mistake=None):
    """items: (n_kv0, n_kv1, N, first edge tile)."""
    sc = Sched(seed)
    item_full, item_empty = [Bar() for _ in range(RING)], [Bar(3) for _ in range(RING)]
    q_full, q_empty = [Bar(), Bar()], [Bar(), Bar()]
    kv_full, kv_empty = [Bar() for _ in range(stages)], [Bar() for _ in range(stages)]
    s_full, p_ready, o_full = [Bar(), Bar()], [Bar(), Bar()], [Bar(), Bar()]
    g_full, g_clean = [Bar() for _ in range(GUARD_RING)], [Bar(2) for _ in range(GUARD_RING)]
    req, ring = [None] * GUARD_RING, [None] * RING
    cleaned_uses = set()
    stream = list(items) + [(0, 0, -1, 0)]

    def producer():
        q_uses, issued, requests = [0, 0], 0, 0
        for k, it in enumerate(stream):
            slot = k % RING
            if k >= RING:
                yield wait(item_empty[slot], k // RING - 1)
            ring[slot] = it
            item_full[slot].arrive()
            if it[2] < 0:
                break

            def load_q(x):
                if it[x] == 0:
                    return
                if q_uses[x] > 0:
                    yield wait(q_empty[x], q_uses[x] - 1)
                sc.tma.append(q_full[x])
                q_uses[x] += 1

            def load_kv(j, kv):
                nonlocal issued, requests
                s = issued % stages
                if issued >= stages:
                    yield wait(kv_empty[s], issued // stages - 1)
                sc.tma.append(kv_full[s])
                if kv and j >= it[3]:
                    assert req[requests % GUARD_RING] is None, "request slot still open"
                    req[requests % GUARD_RING] = (s, issued // stages, issued)
                    g_full[requests % GUARD_RING].arrive()
                    requests += 1
                issued += 1

            yield from load_q(0)
            for j in range(it[2]):
                yield from load_kv(j, 0)
                if j == 0:
                    yield from load_q(1)
                yield from load_kv(j, 1)
        assert req[requests % GUARD_RING] is None, "request slot still open"
        req[requests % GUARD_RING] = (-1, 0, 0)
        g_full[requests % GUARD_RING].arrive()

    def guard(lane):
        r = 0
        while True:
            yield wait(g_full[r % GUARD_RING], r // GUARD_RING)
            s, phase, use = req[r % GUARD_RING]
            if s < 0:
                return
            if mistake == "guard_off_by_a_phase":
                phase += 1
            yield wait_parity(kv_full[s], phase)
            assert kv_full[s].phase == phase + 1, "guard passes over a tile that is not the one requested"
            if lane == 1:
                cleaned_uses.add(use)
            if g_clean[r % GUARD_RING].pending == 1:  # the other warp is done too
                req[r % GUARD_RING] = None
            g_clean[r % GUARD_RING].arrive()
            r += 1

    def mma():
        consumed, cleaned, q_uses, pr = 0, 0, [0, 0], [0, 0]
        for k in range(len(stream)):
            yield wait(item_full[k % RING], k // RING)
            n0, n1, N, edge = ring[k % RING]
            item_empty[k % RING].arrive()
            if N < 0:
                return
            kslot, have_k = 0, False
            for x, n in enumerate((n0, n1)):
                if n == 0:
                    continue
                yield wait(q_full[x], q_uses[x])
                q_uses[x] += 1
                if not have_k:
                    kslot = consumed % stages
                    yield wait(kv_full[kslot], consumed // stages)
                    consumed += 1
                    have_k = True
                sc.commit.append(s_full[x])
                if n == 1:
                    sc.commit.append(q_empty[x])
            sc.commit.append(kv_empty[kslot])
            for j in range(N):
                vslot, use = consumed % stages, consumed
                yield wait(kv_full[vslot], consumed // stages)
                consumed += 1
                if j >= edge:
                    if mistake != "mma_skips_guard":
                        yield wait(g_clean[cleaned % GUARD_RING], cleaned // GUARD_RING)
                    cleaned += 1
                    assert use in cleaned_uses, "edge tile read before it was clean"
                if j < n0:
                    yield wait(p_ready[0], pr[0])
                    pr[0] += 1
                    if j == n0 - 1:
                        sc.commit.append(o_full[0])
                nxt, nslot = j + 1 < N, 0
                if nxt:
                    nslot = consumed % stages
                    yield wait(kv_full[nslot], consumed // stages)
                    consumed += 1
                    if j + 1 < n0:
                        sc.commit.append(s_full[0])
                        if j + 2 == n0:
                            sc.commit.append(q_empty[0])
                if j < n1:
                    yield wait(p_ready[1], pr[1])
                    pr[1] += 1
                    if j == n1 - 1:
                        sc.commit.append(o_full[1])
                sc.commit.append(kv_empty[vslot])
                if nxt:
                    if j + 1 < n1:
                        sc.commit.append(s_full[1])
                        if j + 2 == n1:
                            sc.commit.append(q_empty[1])
                    sc.commit.append(kv_empty[nslot])

    def softmax(x):
        sp, o_uses = 0, 0
        for k in range(len(stream)):
            slot = k % RING
            yield wait(item_full[slot], k // RING)
            it = ring[slot]
            if it[2] < 0:
                item_empty[slot].arrive()
                return
            for _ in range(it[x]):
                yield wait(s_full[x], sp)
                sp += 1
                p_ready[x].arrive()
            if it[x] > 0:
                yield wait(o_full[x], o_uses)
                o_uses += 1
            assert ring[slot] is it, "item ring slot overwritten before it was released"
            item_empty[slot].arrive()

    return sc.run({"producer": producer(), "mma": mma(), "softmax0": softmax(0), "softmax1": softmax(1),
                   "guard0": guard(0), "guard1": guard(1)})


def packed_items(rnd):
    out = []
    for _ in range(rnd.randint(1, 24)):
        N = rnd.choice((1, 1, 1, 2, 3, rnd.randint(1, 9)))
        kind = rnd.random()
        if kind < 0.4:
            out.append((N, N, N, N - 1))                             # two heads, diagonal tile last
        elif kind < 0.7:
            out.append((N - 1, N, N, N - 2) if N > 1 else (1, 0, 1, 0))  # causal pair of tiles
        elif kind < 0.85:
            out.append((N, N, N, rnd.choice((N - 1, N))))            # not causal: ragged end or none
        else:
            out.append((N, 0, N, N - 1))
    return out


def _trials(stages, mistake=None, trials=150):
    rnd = random.Random(stages + 100 * (mistake is not None))
    bad = []
    for t in range(trials):
        items = packed_items(rnd)
        for seed in range(2):
            try:
                r = packed_run(items, stages, seed + 10 * t, mistake)
            except (Hazard, AssertionError) as e:
                r = f"{type(e).__name__}: {e}"
            if r:
                bad.append((t, seed, r, items))
    return bad


@pytest.mark.parametrize("stages", [4, 8])  # the K/V ring at D = 128 and D = 64
def test_packed_protocol(stages):
    bad = _trials(stages)
    assert not bad, bad[:3]


@pytest.mark.parametrize("mistake", ["mma_skips_guard", "guard_off_by_a_phase"])
def test_packed_model_catches_planted_mistakes(mistake):
    assert _trials(4, mistake, trials=60), f"the model missed '{mistake}'"


# ----------------------------------------------------------------------------- tree

def tree_run(runs, stages, seed, mistake=None):
    """runs: (n tiles, first edge tile, one row tile?) per unit run of a CTA."""
    sc = Sched(seed)
    run_full, run_empty = [Bar() for _ in range(RING)], [Bar(3) for _ in range(RING)]
    q_full, q_free, q_first = [Bar(2), Bar(2)], Bar(), Bar(2)
    kv_full, kv_empty = [Bar() for _ in range(stages)], [Bar() for _ in range(stages)]
    s_full, p_ready, o_full = [Bar(), Bar()], [Bar(), Bar()], [Bar(), Bar()]
    g_full, g_clean = [Bar() for _ in range(TREE_REQS)], [Bar(2) for _ in range(TREE_REQS)]
    join = Bar(2)
    req, ring = [None] * TREE_REQS, [None] * RING
    open_reqs = [0]
    cleaned_uses = set()
    staged = {}                # guard warps that have staged a run's Q and sets
    q_owner = [None]           # run whose Q is staged
    set_owner = [None, None]   # run whose ancestor sets are in each buffer
    o_owner = [None, None]     # run whose values O_x accumulates
    stream = list(runs) + [(-1, 0, False)]

    def producer():
        issued, requests = 0, 0
        for k, r in enumerate(stream):
            if k >= RING:
                yield wait(run_empty[k % RING], k // RING - 1)
            ring[k % RING] = r
            run_full[k % RING].arrive()
            n, edge, one = r
            if n < 0:
                break

            def request(what):
                nonlocal requests
                assert req[requests % TREE_REQS] is None, "request slot still open"
                req[requests % TREE_REQS] = what
                g_full[requests % TREE_REQS].arrive()
                requests += 1

            request((-2, 0, k))
            order = [(0, 0), (1, 0)] + [x for j in range(n) for x in ((j, 1), (j + 2, 0))] if one else [
                x for j in range(n) for x in ((j, 0), (j, 1))]
            for i, (j, kv) in enumerate(order):
                if i == 1 and k == 0:
                    yield wait(q_first, 0)
                if j >= n:
                    continue
                s = issued % stages
                if issued >= stages:
                    yield wait(kv_empty[s], issued // stages - 1)
                sc.tma.append(kv_full[s])
                if kv and j >= edge:
                    request((s, issued // stages, issued))
                issued += 1
        assert req[requests % TREE_REQS] is None, "request slot still open"
        req[requests % TREE_REQS] = (-1, 0, 0)
        g_full[requests % TREE_REQS].arrive()

    done = {}

    def guard(lane):
        r, cleaned = 0, 0
        while True:
            yield wait(g_full[r % TREE_REQS], r // TREE_REQS)
            s, phase, use = req[r % TREE_REQS]
            if s == -1:
                return
            if s == -2:
                k = use
                if k >= 2:
                    yield wait(run_empty[(k - 2) % RING], (k - 2) // RING)
                set_owner[k & 1] = k
                if k >= 1:
                    if mistake != "no_q_free":
                        yield wait(q_free, k - 1)
                    staged[k] = staged.get(k, 0) + 1
                    q_owner[0] = k if staged[k] == 2 else None
                q_full[k & 1].arrive()
            else:
                yield wait_parity(kv_full[s], phase)
                assert kv_full[s].phase == phase + 1, "guard passes over a tile that is not the one requested"
                cleaned_uses.add((lane, use))
                g_clean[cleaned % TREE_REQS].arrive()
                cleaned += 1
            done[r] = done.get(r, 0) + 1
            if done[r] == 2:
                req[r % TREE_REQS] = None
            r += 1

    def mma():
        st = dict(consumed=0, cleaned=0)
        pr = [0, 0]

        def stage():
            s, use = st["consumed"] % stages, st["consumed"]
            yield wait(kv_full[s], use // stages)
            st["consumed"] += 1
            st["slot"], st["use"] = s, use

        def v_tile(j, edge):
            yield from stage()
            if j >= edge:
                if mistake != "mma_skips_guard":
                    yield wait(g_clean[st["cleaned"] % TREE_REQS], st["cleaned"] // TREE_REQS)
                st["cleaned"] += 1
                assert {(0, st["use"]), (1, st["use"])} <= cleaned_uses, "edge tile read before it was clean"
            return st["slot"]

        def scores(x, k, left):
            assert q_owner[0] == k, "Q of another run"
            sc.commit.append(s_full[x])
            left[0] -= 1
            if left[0] == 0:
                sc.commit.append(q_free)

        def mix(x, k):
            assert o_owner[x] in (None, k), "O still belongs to another run"
            o_owner[x] = k

        for k in range(len(stream)):
            yield wait(run_full[k % RING], k // RING)
            n, edge, one = ring[k % RING]
            run_empty[k % RING].arrive()
            if n < 0:
                return
            yield wait(*((q_first, 0) if k == 0 else (q_full[k & 1], k >> 1)))
            left = [(2 * n if not one else n)]  # S MMAs of the run still to issue
            if one:
                for x in range(min(2, n)):
                    yield from stage()
                    scores(x, k, left)
                    sc.commit.append(kv_empty[st["slot"]])
                for j in range(n):
                    x = j & 1
                    vs = yield from v_tile(j, edge)
                    yield wait(p_ready[x], pr[x])
                    pr[x] += 1
                    mix(x, k)
                    if j + 2 >= n:
                        sc.commit.append(o_full[x])
                    sc.commit.append(kv_empty[vs])
                    if j + 2 < n:
                        yield from stage()
                        scores(x, k, left)
                        sc.commit.append(kv_empty[st["slot"]])
            else:
                yield from stage()
                ks = st["slot"]
                scores(0, k, left)
                scores(1, k, left)
                sc.commit.append(kv_empty[ks])
                for j in range(n):
                    vs = yield from v_tile(j, edge)
                    yield wait(p_ready[0], pr[0])
                    pr[0] += 1
                    mix(0, k)
                    if j + 1 == n:
                        sc.commit.append(o_full[0])
                    else:
                        yield from stage()
                        ks = st["slot"]
                        scores(0, k, left)
                    yield wait(p_ready[1], pr[1])
                    pr[1] += 1
                    mix(1, k)
                    if j + 1 == n:
                        sc.commit.append(o_full[1])
                    sc.commit.append(kv_empty[vs])
                    if j + 1 < n:
                        scores(1, k, left)
                        sc.commit.append(kv_empty[ks])

    def softmax(x):
        sp, o_uses, joins = 0, [0, 0], 0
        for k in range(len(stream)):
            yield wait(run_full[k % RING], k // RING)
            r = ring[k % RING]
            n, edge, one = r
            if n < 0:
                return
            if k == 0:
                staged[0] = staged.get(0, 0) + 1
                q_owner[0] = 0 if staged[0] == 2 else None
                q_first.arrive()
            yield wait(q_full[k & 1], k >> 1)
            for _ in range((n - x + 1) // 2 if one else n):
                yield wait(s_full[x], sp)
                sp += 1
                assert set_owner[k & 1] == k, "ancestor sets of another run"
                p_ready[x].arrive()
            if one:
                join.arrive()
                yield wait(join, joins)
                joins += 1
            for y in range(2):
                used = not one or y < n
                if used and (one or y == x):
                    yield wait(o_full[y], o_uses[y])
                o_uses[y] += used
            for y in range(2):
                if (not one and y == x) or (one and y < n):
                    assert o_owner[y] == k, "O overwritten before it was read"
            assert ring[k % RING] is r, "run slot overwritten before it was released"
            assert set_owner[k & 1] == k, "ancestor sets of another run"
            run_empty[k % RING].arrive()
            o_owner[x] = None if not one else o_owner[x]
            if one and mistake != "no_join":
                join.arrive()
                yield wait(join, joins)
                joins += 1
            o_owner[x] = None

    return sc.run({"producer": producer(), "mma": mma(), "softmax0": softmax(0), "softmax1": softmax(1),
                   "guard0": guard(0), "guard1": guard(1)})


def _tree_trials(stages, mistake=None, trials=200):
    rnd = random.Random(stages + 17 * (mistake is not None))
    bad = []
    for t in range(trials):
        runs = []
        for _ in range(rnd.randint(1, 10)):
            n = rnd.choice((1, 1, 2, 3, rnd.randint(1, 12)))
            runs.append((n, max(0, n - rnd.randint(0, 3)), stages == 5 or rnd.random() < 0.5))
        for seed in range(2):
            try:
                r = tree_run(runs, stages, seed + 10 * t, mistake)
            except (Hazard, AssertionError) as e:
                r = f"{type(e).__name__}: {e}"
            if r:
                bad.append((t, seed, r, runs))
    return bad


@pytest.mark.parametrize("stages", [4, 5, 8])  # pairs and single row tiles at D = 128, both at D = 64
def test_tree_protocol(stages):
    bad = _tree_trials(stages)
    assert not bad, bad[:3]


@pytest.mark.parametrize("mistake", ["mma_skips_guard", "no_join", "no_q_free"])
def test_tree_model_catches_planted_mistakes(mistake):
    assert _tree_trials(4, mistake, trials=80), f"the model missed '{mistake}'"
