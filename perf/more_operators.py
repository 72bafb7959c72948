"""Timing cases of a paged KV cache, each in a plain torch form and as the library's calls.

    paged    attention of new tokens (chunks of prompts, single tokens, both together) over a paged cache (attn_fwd_paged)
    norm     RMS norm of each head row of q and k with the rotary turn (attn_norm_rope), and that with the append of keys
             and values to their pages (attn_rope_append_paged)
    pages    the table of pages: growing, cutting back and forking sequences (attn_pages_step), moving pages together
             (attn_pages_compact), and the copies of pages that these ask for (attn_pages_copy)

``own`` selects which form ``run`` takes.  Values are i.i.d. N(0, 1) drawn on the device from the seed, as in the library's
workloads; sizes (lengths, forks) belong to the case; which page holds what follows from the seed.  Head counts and depths are
those of the library's workloads: 32 query heads with 32 or 8 key/value heads of depth 128, 4 heads of depth 64 in fp32.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    gqa = dict(H=32, Hkv=8, D=128, dtype="bf16")
    small = dict(H=4, Hkv=2, D=64, dtype="f32")
    return [
        # a decode step of one user: latency counts
        dict(name="paged one user", op="paged", B=1, low=1501, high=1501, sizes=1, chunks="", P=16, lse=False, **gqa),
        # a decode step of a full batch, one token each
        dict(name="paged decode batch", op="paged", B=64, low=1, high=8192, sizes=2, chunks="", P=64, lse=False, **gqa),
        # the same with a cached head for each query head
        dict(name="paged decode all heads", op="paged", B=16, low=100, high=4096, sizes=3, chunks="", P=16, lse=False,
             **dict(gqa, Hkv=32)),
        # a step of a server that mixes decoding sequences with chunks of prompts (new tokens:tokens in the cache)
        dict(name="paged mixed step", op="paged", B=60, low=200, high=6000, sizes=4, chunks="512:0,512:1536,300:5003,77:0",
             P=32, lse=False, **gqa),
        # a chunk of a long document
        dict(name="paged long chunk", op="paged", B=0, low=0, high=0, sizes=5, chunks="4096:28672", P=128, lse=True, **gqa),
        # fp32
        dict(name="paged f32", op="paged", B=6, low=1, high=1024, sizes=6, chunks="100:57,33:0", P=16, lse=True, **small),
        # one decode step: each of 64 sequences appends one token
        dict(name="norm append step", op="append", lens=",".join(["1"] * 64), past=700, P=16, layout="half", rotary=128,
             scaling="none", normed=True, **gqa),
        # prompts into the pages, frequencies scaled for long contexts
        dict(name="norm append prompts", op="append", lens="8192,4096,2050,1025,511,300,200,11", past=0, P=64, layout="half",
             rotary=128, scaling="wavelength", normed=True, **gqa),
        # an encoder's norm and turn without a cache, a rotary depth that is no multiple of 16
        dict(name="norm rope f32", op="norm", T=2055, far=4096, layout="interleaved", rotary=36, scaling="none", **dict(small, Hkv=4)),
        # the table of a large server over one decode step
        dict(name="pages step", op="step", users=256, beams=1, low=16, high=7000, sizes=7, P=16, M=512, spare=1.2, layers=0,
             cut=0, grow=1, **gqa),
        # a step of beam search: every user's beams go on from some of them, partly filled pages are copied
        dict(name="pages fork beams", op="step", users=32, beams=4, low=100, high=600, sizes=8, P=32, M=64, spare=1.5, layers=4,
             cut=0, grow=1, **gqa),
        # a half empty pool is moved together
        dict(name="pages compact", op="compact", users=64, beams=1, low=16, high=2048, sizes=9, P=16, M=160, spare=2.0, layers=1,
             **gqa),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    if rng.random() < 0.2:
        return dict(H=4, Hkv=rng.choice((1, 2, 4)), D=64, dtype="f32")
    return dict(H=rng.choice((16, 32)), Hkv=rng.choice((1, 2, 8, 16)), D=rng.choice((64, 128)), dtype="bf16")


def draw(rng):
    op = rng.choice(("paged", "paged", "paged", "append", "norm", "step", "compact"))
    h = _heads(rng)
    f32 = h["dtype"] == "f32"
    P = rng.choice((8, 16, 32, 64, 128, 256))
    sizes = rng.randrange(1 << 30)
    if op == "paged":
        high = _log(rng, 8, 2048 if f32 else 8192)
        B = _log(rng, 1, 64)
        chunks = []
        if rng.random() < 0.6:
            for _ in range(rng.randint(1, 4)):
                chunks.append("%d:%d" % (_log(rng, 2, 256 if f32 else 2048), rng.choice((0, _log(rng, 1, 1024 if f32 else 12000)))))
            B = rng.choice((0, B))
        return dict(op=op, B=B, low=max(1, high // rng.randint(1, 100)), high=high, sizes=sizes, chunks=",".join(chunks), P=P,
                    lse=rng.random() < 0.5, **h)
    turn = dict(layout=rng.choice(("half", "interleaved")), scaling=rng.choice(("none", "linear", "wavelength")),
                rotary=2 * rng.randint(1, h["D"] // 2) if rng.random() < 0.3 else rng.choice((h["D"], h["D"] // 2)))
    if op == "append":
        n = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, 16000 // n))
        lens = [longest] + [_log(rng, 1, longest) for _ in range(n - 1)]
        rng.shuffle(lens)
        return dict(op=op, lens=",".join(map(str, lens)), past=_log(rng, 1, 2000), P=P, normed=rng.random() < 0.7, **turn, **h)
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 16384), far=_log(rng, 1, 2000000), **turn, **h)
    users, beams = _log(rng, 1, 128), rng.choice((1, 1, 2, 4)) if op == "step" else 1
    high = _log(rng, 8, max(8, min(4096, 65536 // (users * beams))))
    c = dict(op=op, users=users, beams=beams, low=max(1, high // 8), high=high, sizes=sizes, P=P,
             M=(high + 64) // P + rng.randint(2, 40), spare=rng.choice((1.2, 1.5, 2.0)), layers=rng.choice((0, 1, 2)), **h)
    return dict(c, cut=rng.choice((0, 0, 20)), grow=_log(rng, 1, 64)) if op == "step" else c


# ------------------------------------------------------------------ sizes of a case

def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _sequences(case):
    """(tokens in the cache before, new tokens) of each sequence of a paged case."""
    r = random.Random(case["sizes"])
    seqs = [(r.randint(case["low"], case["high"]) - 1, 1) for _ in range(case["B"])]
    for c in filter(None, case["chunks"].split(",")):
        new, past = c.split(":")
        seqs.append((int(past), int(new)))
    r.shuffle(seqs)
    return seqs


def _forks(case):
    """(length before, parent, length after) of each row of a step or compact case."""
    r = random.Random(case["sizes"])
    rows = []
    for u in range(case["users"]):
        L = r.randint(case["low"], case["high"])
        for _ in range(case["beams"]):
            parent = u * case["beams"] + r.randrange(case["beams"])
            new = L + case.get("grow", 0) if r.random() < 0.9 else max(0, L - r.randint(0, case.get("cut", 0)))
            rows.append((L, parent, new))
    return rows


def _frequencies(case):
    """Rotary frequencies (radians per position), scaled as the case says."""
    r = case["rotary"]
    w = [10000.0 ** (-2.0 * p / r) for p in range(r // 2)]
    if case["scaling"] == "linear":
        w = [x / 8.0 for x in w]
    if case["scaling"] == "wavelength":
        turns = [8192 * x / (2 * math.pi) for x in w]  # turns over the original context
        w = [x / 8.0 if t < 1.0 else x if t > 4.0 else x * ((1 - (t - 1) / 3) / 8.0 + (t - 1) / 3) for x, t in zip(w, turns)]
    return w


def _used_pages(case):
    """Pages held by the rows of a step or compact case: a user's beams share the full ones."""
    P, beams = case["P"], case["beams"]
    lens = [L for L, _, _ in _forks(case)][::beams]
    return sum(L // P + (beams if L % P else 0) for L in lens)


def work(case):
    H, Hkv, D, e = case["H"], case["Hkv"], case["D"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "paged":
        seqs = _sequences(case)
        T, held = sum(n for _, n in seqs), sum(p + n for p, n in seqs)
        pairs = sum(n * p + n * (n + 1) // 2 for p, n in seqs)
        return {"bytes": 2 * T * H * D * e + 2 * held * Hkv * D * e + 4 * held // case["P"], "flops": 4 * D * H * pairs}
    if case["op"] in ("append", "norm"):
        append = case["op"] == "append"
        T = sum(_lens(case)) if append else case["T"]
        norm = 4 * D * T * (H + Hkv) if not append or case["normed"] else 0
        return {"bytes": 2 * T * (H + (2 if append else 1) * Hkv) * D * e + 4 * T,
                "flops": norm + 3 * T * (H + Hkv) * case["rotary"]}
    rows, P = _forks(case), case["P"]
    page = 2 * case["layers"] * Hkv * D * e  # bytes of one row of a page, k and v, in all layers
    used = _used_pages(case)
    if case["op"] == "step":
        entries = sum(min(rows[p][0], new) // P for _, p, new in rows)
        first, copied = set(), 0
        for _, p, new in rows:
            kept = min(rows[p][0], new)
            if kept % P and p in first:
                copied += kept % P
            first.add(p)
        return {"bytes": 4 * entries + 4 * len(rows) * case["M"] + 2 * copied * page, "flops": entries}
    moved = used * (1.0 - 1.0 / case["spare"])  # on average, pages lying at random
    return {"bytes": int(8 * len(rows) * case["M"] + 2 * moved * P * page), "flops": used}


# ------------------------------------------------------------------ inputs

def _tables(rng, counts, M, n_pages):
    """A table of M entries a row whose first counts[b] name distinct pages; what stands behind them is left over."""
    ids = rng.permutation(n_pages).astype(np.int32)
    table = rng.integers(0, n_pages, (len(counts), M), dtype=np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    H, Hkv, D, P = case["H"], case["Hkv"], case["D"], case.get("P", 0)

    def normal(*shape):
        # in parts: the 32-bit draws of a large pool need not fit beside it
        out = torch.empty(shape, dtype=dt, device="cuda")
        for part in out.view(-1).split(1 << 28):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.float32))
        return out

    def ints(v):
        return torch.as_tensor(np.asarray(v, dtype=np.int32)).cuda()

    s = dict(case=dict(case))
    if case["op"] in ("paged", "append"):
        seqs = _sequences(case) if case["op"] == "paged" else [(case["past"], n) for n in _lens(case)]
        counts = [-(-(p + n) // P) for p, n in seqs]
        n_pages = sum(counts) + sum(counts) // 8 + 2
        ends = [sum(n for _, n in seqs[:i]) for i in range(len(seqs) + 1)]
        T = ends[-1]
        s.update(kpages=normal(n_pages, Hkv, P, D), vpages=normal(n_pages, Hkv, P, D),
                 table=ints(_tables(rng, counts, max(counts) + 3, n_pages)), cache_len=ints([p + n for p, n in seqs]),
                 cu_seqlens=ints(ends) if T != len(seqs) else None, seqs=seqs, ends=ends)
        if case["op"] == "paged":
            s["q"] = normal(T, H, D)
        else:  # one projection writes q, k and v side by side; the call takes its slices
            qkv = normal(T, H + 2 * Hkv, D)
            s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
    if case["op"] == "norm":
        s.update(q=normal(case["T"], H, D), k=normal(case["T"], Hkv, D),
                 positions=torch.randint(0, case["far"], (case["T"],), generator=g, device="cuda").to(torch.int32))
    if case["op"] in ("append", "norm"):
        s["freqs"] = torch.tensor(_frequencies(case), dtype=torch.float64)
        s["weights"] = [(1.0 + 0.1 * normal(D)).to(dt) for _ in range(2)] if case.get("normed", True) else [None, None]
        s["eps"] = 1e-6
    if case["op"] in ("step", "compact"):
        rows, beams = _forks(case), case["beams"]
        used = _used_pages(case)
        n_pages = int(used * case["spare"]) + len(rows) * (2 + case.get("grow", 0) // P) + 1
        table = np.full((len(rows), case["M"]), -1, dtype=np.int32)
        ids, at = rng.permutation(n_pages).astype(np.int32), 0
        for u in range(case["users"]):
            L = rows[u * beams][0]
            shared = ids[at:at + L // P]
            at += L // P
            for b in range(u * beams, (u + 1) * beams):
                table[b, :L // P] = shared
                if L % P:
                    table[b, L // P] = ids[at]
                    at += 1
        s.update(table=ints(table), cache_len=ints([L for L, _, _ in rows]), n_pages=n_pages)
        if case["op"] == "step":
            s.update(parents=ints([p for _, p, _ in rows]) if beams > 1 else None, new_len=ints([n for _, _, n in rows]))
        if case["layers"]:
            s.update(kpages=normal(case["layers"], n_pages, Hkv, P, D), vpages=normal(case["layers"], n_pages, Hkv, P, D))
    return s


# ------------------------------------------------------------------ plain forms

def _attend_plain(q, k, v, seen, out_dtype):
    """q (n, Hkv, R, D), k and v (n, Hkv, L, D) in 32 bits, seen (n, 1, R, L): (out, log of the sum)."""
    x = torch.matmul(q, k.transpose(2, 3))
    x *= 1.0 / math.sqrt(q.shape[-1])
    x.masked_fill_(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True)
    x -= m
    x.exp_()
    total = x.sum(-1, keepdim=True)
    return (torch.matmul(x, v) / total).to(out_dtype), (m + total.log())[..., 0]


def _paged_plain(s):
    case = s["case"]
    q, P, Hkv = s["q"], case["P"], case["Hkv"]
    T, H, D = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    table = s["table"].long()
    ones = [i for i, (_, n) in enumerate(s["seqs"]) if n == 1]
    if ones:  # single tokens side by side, padded to the longest
        longest = max(s["seqs"][i][0] + 1 for i in ones)
        row = torch.tensor(ones, device=q.device)
        at = torch.tensor([s["ends"][i] for i in ones], device=q.device)
        pages = table[row, :-(-longest // P)]
        seen = torch.arange(pages.shape[1] * P, device=q.device) < s["cache_len"].long()[row][:, None]
        k, v = (x[pages].transpose(1, 2).flatten(2, 3).float() for x in (s["kpages"], s["vpages"]))
        o, l = _attend_plain(q[at].float().view(len(ones), Hkv, H // Hkv, D), k, v, seen[:, None, None], q.dtype)
        out[at], lse[at] = o.view(-1, H, D), l.view(-1, H)
    for i, (past, n) in enumerate(s["seqs"]):
        if n == 1:
            continue
        rows, L = slice(s["ends"][i], s["ends"][i + 1]), past + n
        pages = table[i, :-(-L // P)]
        k, v = (x[pages].transpose(0, 1).flatten(1, 2)[:, :L] for x in (s["kpages"], s["vpages"]))
        seen = torch.arange(L, device=q.device) <= past + torch.arange(n, device=q.device)[:, None]
        seen = seen.repeat(H // Hkv, 1)[None, None]
        for h in range(Hkv):  # one head after the other: the scores of all would not fit
            heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            qh = q[rows, heads].float().transpose(0, 1).reshape(1, 1, -1, D)
            o, l = _attend_plain(qh, k[None, h:h + 1].float(), v[None, h:h + 1].float(), seen, q.dtype)
            out[rows, heads] = o.view(-1, n, D).transpose(0, 1)
            lse[rows, heads] = l.view(-1, n).T
    return (out, lse) if case["lse"] else out


def _norm_plain(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _turn_plain(x, positions, freqs, rotary, layout):
    angle = positions.double()[:, None] * freqs.to(x.device)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, rest = x[..., :rotary], x[..., rotary:]
    if layout == "half":
        a, b = rot[..., :rotary // 2], rot[..., rotary // 2:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((rot, rest), dim=-1)


def _append_plain(s):
    case, P = s["case"], s["case"]["P"]
    q, k, v, lens = s["q"], s["k"], s["v"], s["cache_len"].long()
    t = torch.arange(q.shape[0], device=q.device)
    if s["cu_seqlens"] is None:
        seq, row = t, lens - 1
    else:
        cu = s["cu_seqlens"].long()
        seq = (t[:, None] >= cu[None, 1:]).sum(1)
        row = lens[seq] - (cu[seq + 1] - t)
    page, at = s["table"].long()[seq, row // P], row % P
    turn = (row, s["freqs"], case["rotary"], case["layout"])
    s["kpages"][page, :, at] = _turn_plain(_norm_plain(k, s["weights"][1], s["eps"]), *turn).to(k.dtype)
    s["vpages"][page, :, at] = v
    return _turn_plain(_norm_plain(q, s["weights"][0], s["eps"]), *turn).to(q.dtype), s["kpages"], s["vpages"]


def _step_plain(table, lens, n_pages, P, parents, new_len):
    """The next table: row b goes on from row parents[b], cut or grown to new_len[b] tokens.  A full page is shared, a partly
    filled one has one holder: its first, unless another row holds it as a full one; the others get a copy.  New pages are the
    lowest free ones, in the order of rows and entries."""
    B, M = table.shape
    dev = table.device
    old, L = table.long(), lens.long()
    if parents is not None:
        old, L = old[parents.long()], L[parents.long()]
    new = new_len.long().clamp(0, M * P)
    keep = torch.minimum(L, new)
    full, part = keep // P, keep % P
    i = torch.arange(M, device=dev)
    in_full = i < full[:, None]
    held = torch.zeros(n_pages, dtype=torch.bool, device=dev)
    held[old[in_full]] = True
    b = torch.arange(B, device=dev)
    last = old.gather(1, full.clamp(max=M - 1)[:, None])[:, 0].clamp(0, n_pages - 1)  # the partly filled page
    first = torch.full((n_pages,), B, device=dev)
    first.scatter_reduce_(0, last, torch.where(part > 0, b, B), "amin")
    stays = (part > 0) & ~held[last] & (first[last] == b)
    held[last[stays]] = True
    kept = full + stays
    free = ~held
    rank = free.long().cumsum(0) - 1
    order = torch.empty(n_pages, dtype=torch.long, device=dev)
    order[rank[free]] = torch.arange(n_pages, device=dev)[free]
    count = free.sum()
    wanted = (i >= kept[:, None]) & (i < ((new + P - 1) // P)[:, None])
    nth = (wanted.flatten().long().cumsum(0) - 1).view(B, M)
    given = torch.where(nth < count, order[nth.clamp(0, n_pages - 1)], -1)
    out = torch.where(i < kept[:, None], old, torch.where(wanted, given, -1))
    to = out.gather(1, full.clamp(max=M - 1)[:, None])[:, 0]
    copied = (part > 0) & ~stays & (to >= 0)
    copies = torch.stack((last, to, part), 1)
    copies = torch.where(copied[:, None], copies, torch.tensor([-1, -1, 0], device=dev))
    return (out.to(torch.int32), new.to(torch.int32), copies.to(torch.int32),
            (count - wanted.sum()).to(torch.int32).view(1))


def _compact_plain(table, lens, n_pages, P):
    """The held pages moved to the front: the lowest held page behind the first n (n pages are held) to the lowest free one."""
    B, M = table.shape
    dev = table.device
    i = torch.arange(M, device=dev)
    mine = i < ((lens.long() + P - 1) // P)[:, None]
    held = torch.zeros(n_pages, dtype=torch.bool, device=dev)
    held[table.long()[mine]] = True
    n = held.sum()
    p = torch.arange(n_pages, device=dev)
    hole, moved = ~held & (p < n), held & (p >= n)
    copies = torch.tensor([-1, -1, 0], device=dev).repeat((n_pages + 1) // 2, 1)
    to_hole, of_moved = (torch.empty(n_pages, dtype=torch.long, device=dev) for _ in range(2))
    to_hole[(hole.long().cumsum(0) - 1)[hole]] = p[hole]
    rank = moved.long().cumsum(0) - 1
    of_moved[rank[moved]] = p[moved]
    c = torch.arange(copies.shape[0], device=dev)
    some = c < moved.sum()
    copies = torch.where(some[:, None], torch.stack((of_moved[c], to_hole[c], torch.full_like(c, P)), 1), copies)
    where = torch.where(moved, to_hole[rank.clamp(min=0)], p)
    out = torch.where(mine, where[table.long().clamp(0, n_pages - 1)], -1)
    return out.to(torch.int32), copies.to(torch.int32), (n_pages - n).to(torch.int32).view(1)


def _copy_plain(kpages, vpages, copies):
    src, dst, rows = copies[copies[:, 0] >= 0].long().unbind(1)
    some = (torch.arange(kpages.shape[3], device=kpages.device) < rows[:, None])[None, :, None, :, None]
    for x in (kpages, vpages):
        x[:, dst] = torch.where(some, x[:, src], x[:, dst])


def run(s):
    case = s["case"]
    if own:
        import transformer_scaled_dot_fwd_gb300 as attn

        if case["op"] == "paged":
            return attn.attn_fwd_paged(s["q"], s["kpages"], s["vpages"], s["table"], s["cache_len"],
                                       cu_seqlens=s["cu_seqlens"], return_lse=case["lse"])
        if case["op"] == "norm":
            return attn.attn_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], *s["weights"], eps=s["eps"],
                                       interleaved=case["layout"] == "interleaved")
        if case["op"] == "append":
            q = attn.attn_rope_append_paged(s["q"], s["k"], s["v"], s["kpages"], s["vpages"], s["table"], s["freqs"],
                                            s["cache_len"], cu_seqlens=s["cu_seqlens"], q_weight=s["weights"][0],
                                            k_weight=s["weights"][1], eps=s["eps"], interleaved=case["layout"] == "interleaved")
            return q, s["kpages"], s["vpages"]
        if case["op"] == "step":
            table, lens, copies, free = attn.attn_pages_step(s["table"], s["cache_len"], s["n_pages"], case["P"],
                                                             parents=s["parents"], new_len=s["new_len"])
            r = table, lens, copies, free
        else:
            table, copies, free = r = attn.attn_pages_compact(s["table"], s["cache_len"], s["n_pages"], case["P"])
        if not case["layers"]:
            return r
        attn.attn_pages_copy(s["kpages"], s["vpages"], copies)
        return (*r, s["kpages"], s["vpages"])
    if case["op"] == "paged":
        return _paged_plain(s)
    if case["op"] == "norm":
        turn = (s["positions"], s["freqs"], case["rotary"], case["layout"])
        return tuple(_turn_plain(_norm_plain(x, w, s["eps"]), *turn).to(x.dtype) for x, w in zip((s["q"], s["k"]), s["weights"]))
    if case["op"] == "append":
        return _append_plain(s)
    if case["op"] == "step":
        r = _step_plain(s["table"], s["cache_len"], s["n_pages"], case["P"], s["parents"], s["new_len"])
        copies = r[2]
    else:
        r = _compact_plain(s["table"], s["cache_len"], s["n_pages"], case["P"])
        copies = r[1]
    if not case["layers"]:
        return r
    _copy_plain(s["kpages"], s["vpages"], copies)
    return (*r, s["kpages"], s["vpages"])


# ------------------------------------------------------------------ from the definition, in 64 bits

def _turned(x, position, case, weight, eps):
    """Head rows of x (T, heads, D), divided by their root mean square, times the weight; every pair then as a complex number,
    turned by position * frequency."""
    r = case["rotary"]
    x = x.double()
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * weight.double()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
    else:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous())
    w = torch.tensor(_frequencies(case), dtype=torch.float64, device=x.device)
    angle = position.double()[:, None, None] * w
    z = z * torch.polar(torch.ones_like(angle), angle)
    out = x.clone()
    if case["layout"] == "half":
        out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
    else:
        out[..., :r] = torch.view_as_real(z).flatten(-2)
    return out


def exact(case, seed):
    if case["op"] in ("step", "compact"):
        return None  # whole numbers, and copies
    s = prepare(case, seed)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] == "norm":
        return tuple(_turned(x, s["positions"], case, w, s["eps"]) for x, w in zip((s["q"], s["k"]), s["weights"]))
    P, table = case["P"], s["table"].cpu().tolist()
    if case["op"] == "append":
        q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        kp, vp = s["kpages"].double(), s["vpages"].double()
        for i, (past, n) in enumerate(s["seqs"]):
            rows = slice(s["ends"][i], s["ends"][i + 1])
            position = torch.arange(past, past + n, device="cuda")
            q[rows] = _turned(s["q"][rows], position, case, s["weights"][0], s["eps"])
            k = _turned(s["k"][rows], position, case, s["weights"][1], s["eps"])
            v = s["v"][rows].double()
            done = 0
            while done < n:  # page by page
                at = (past + done) % P
                some = min(P - at, n - done)
                page = table[i][(past + done) // P]
                kp[page, :, at:at + some] = k[done:done + some].transpose(0, 1)
                vp[page, :, at:at + some] = v[done:done + some].transpose(0, 1)
                done += some
        return q, kp, vp
    if 4 * D * H * sum(n * p + n * n // 2 for p, n in s["seqs"]) > 6e12:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (past, n) in enumerate(s["seqs"]):
        rows, L = slice(s["ends"][i], s["ends"][i + 1]), past + n
        pages = torch.tensor(table[i][:-(-L // P)], device="cuda")
        j = torch.arange(L, device="cuda")
        hidden = j > past + torch.arange(n, device="cuda")[:, None]
        for g in range(Hkv):
            k = s["kpages"][pages, g].double().reshape(-1, D)[:L]
            v = s["vpages"][pages, g].double().reshape(-1, D)[:L]
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                x = s["q"][rows, h].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                lse[rows, h] = torch.logsumexp(x, -1)
                out[rows, h] = torch.exp(x - lse[rows, h, None]) @ v
    return (out, lse) if case["lse"] else out
