"""Timing cases of three groups of calls, each in a plain torch form and as the library's calls.

    packed   causal or full attention over packed sequences of different lengths (attn_fwd_packed)
    rope     rotary positions in place of a copy, and their append to a KV cache (attn_rope, attn_rope_append)
    tree     attention of a tree of drafted tokens over a KV cache (attn_decode_tree)

``own`` selects which form ``run`` takes.  Inputs are i.i.d. N(0, 1) drawn on the device from the seed, as in the
library's workloads; sizes (lengths, trees) belong to the case.  Head counts and depths are those of the library's
workloads: 32 query heads with 32, 8 or 1 key/value heads of depth 128, 4 heads of depth 64 in fp32.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    gqa = dict(H=32, Hkv=8, D=128, dtype="bf16")
    return [
        # a few short chat turns prefilled together: latency counts
        dict(name="packed chat turns", op="packed", lens="96,17,1,64,33,40", causal=True, **gqa),
        # a serving batch of prompts of mixed lengths, an empty slot among them
        dict(name="packed mixed prompts", op="packed", causal=True, **gqa,
             lens="2048,1531,1024,977,0,700,513,512,400,391,256,255,199,128,127,100,64,63,50,33,31,7,2,1"),
        # long documents
        dict(name="packed documents", op="packed", lens="8192,5001,4097,1023", causal=True, **gqa),
        # fp32 encoder batch: every token sees its whole sequence
        dict(name="packed encoder f32", op="packed", lens="700,513,260,129,64,1", causal=False, H=4, Hkv=4, D=64,
             dtype="f32"),
        # one decode step: each of 64 sequences rotates and appends one token
        dict(name="rope append step", op="append", lens=",".join(["1"] * 64), past="700", Skv=1024, layout="half",
             rotary=128, scaling="none", **gqa),
        # prompts into the cache, frequencies scaled for long contexts
        dict(name="rope append prompts", op="append", lens="8192,4096,2050,1025,511,300,200,11", past="0", Skv=8192,
             layout="half", rotary=128, scaling="wavelength", **gqa),
        # half of the head rotated, neighbouring elements paired, far positions
        dict(name="rope partial far", op="rope", T=32768, far=1000000, layout="interleaved", rotary=64, scaling="linear",
             inverse=False, H=32, Hkv=32, D=128, dtype="bf16"),
        # the rotation's gradient in fp32, a rotary depth that is no multiple of 16
        dict(name="rope inverse f32", op="rope", T=2055, far=4096, layout="half", rotary=36, scaling="none", inverse=True,
             H=4, Hkv=4, D=64, dtype="f32"),
        # one user, a small tree
        dict(name="tree one user", op="tree", B=1, T=8, Skv=2048, low=1500, high=1500, tree=1, ragged=False, **gqa),
        # a batch of users, trees of different sizes
        dict(name="tree batch", op="tree", B=16, T=24, Skv=8192, low=2000, high=8192, tree=2, ragged=True, **gqa),
        # a full machine with wide trees
        dict(name="tree wide batch", op="tree", B=64, T=63, Skv=8192, low=4096, high=8192, tree=3, ragged=False, **gqa),
        # fp32
        dict(name="tree f32", op="tree", B=4, T=13, Skv=1024, low=100, high=1024, tree=4, ragged=True, H=4, Hkv=2, D=64,
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    if rng.random() < 0.25:
        H = 4
        return dict(H=H, Hkv=rng.choice((1, 2, 4)), D=64, dtype="f32")
    H = rng.choice((16, 32))
    return dict(H=H, Hkv=rng.choice((1, 2, 8, 16)), D=rng.choice((64, 128)), dtype="bf16")


def draw(rng):
    op = rng.choice(("packed", "packed", "append", "rope", "tree", "tree"))
    h = _heads(rng)
    f32 = h["dtype"] == "f32"
    layout = rng.choice(("half", "interleaved"))
    scaling = rng.choice(("none", "linear", "ntk", "wavelength"))
    rotary = 2 * rng.randint(1, h["D"] // 2) if rng.random() < 0.4 else rng.choice((h["D"], h["D"] // 2))
    if op == "packed":
        longest = _log(rng, 32, 1024 if f32 else 6000)
        n = _log(rng, 1, max(1, min(48, 60000000 // longest ** 2)))  # the padded plain form costs n * longest^2
        lens = [longest] + [_log(rng, 1, longest) for _ in range(n - 1)]
        rng.shuffle(lens)
        return dict(op=op, lens=",".join(map(str, lens)), causal=rng.random() < 0.75, **h)
    if op == "append":
        n = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, 16000 // n))
        past = _log(rng, 1, 2000)
        lens = [longest] + [_log(rng, 1, longest) for _ in range(n - 1)]
        rng.shuffle(lens)
        return dict(op=op, lens=",".join(map(str, lens)), past=str(past), Skv=past + longest + rng.randint(0, 64),
                    layout=layout, rotary=rotary, scaling=scaling, **h)
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 32768), far=_log(rng, 1, 2000000), layout=layout, rotary=rotary, scaling=scaling,
                    inverse=rng.random() < 0.5, **h)
    B = _log(rng, 1, 48)
    Skv = _log(rng, 200, 4096 if f32 else 8192)
    return dict(op=op, B=B, T=_log(rng, 1, 64), Skv=Skv, low=max(128, Skv // rng.randint(1, 8)), high=Skv,
                tree=rng.randrange(1 << 30), ragged=rng.random() < 0.5, **h)


# ------------------------------------------------------------------ sizes of a case

def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _tree(case):
    """(cache lengths, draft lengths, parents per sequence) of a tree case."""
    r = random.Random(case["tree"])
    cache = [r.randint(case["low"], case["high"]) for _ in range(case["B"])]
    draft = [r.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(case["B"])]
    # a child hangs under one of the last few tokens, now and then at the root
    parents = [[-1 if i == 0 or r.random() < 0.1 else r.randint(max(0, i - 8), i - 1) for i in range(case["T"])]
               for _ in range(case["B"])]
    return cache, draft, parents


def _frequencies(case):
    """Rotary frequencies (radians per position), scaled as the case says."""
    r = case["rotary"]
    theta, factor = 10000.0, 8.0
    if case["scaling"] == "ntk" and r > 2:
        theta *= factor ** (r / (r - 2))
    w = [theta ** (-2.0 * p / r) for p in range(r // 2)]
    if case["scaling"] == "linear":
        w = [x / factor for x in w]
    if case["scaling"] == "wavelength":
        turns = [8192 * x / (2 * math.pi) for x in w]  # turns over the original context
        w = [x / factor if t < 1.0 else x if t > 4.0 else x * ((1 - (t - 1) / 3) / factor + (t - 1) / 3)
             for x, t in zip(w, turns)]
    return w


def work(case):
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "packed":
        lens = _lens(case)
        T = sum(lens)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": 2 * T * (H + Hkv) * D * e + 4 * T * H, "flops": 4 * D * H * pairs}
    if case["op"] in ("append", "rope"):
        T = sum(_lens(case)) if case["op"] == "append" else case["T"]
        rows = H + Hkv + (Hkv if case["op"] == "append" else 0)
        return {"bytes": 2 * T * rows * D * e + 4 * T, "flops": 3 * T * (H + Hkv) * case["rotary"]}
    cache, draft, parents = _tree(case)
    pairs = 0
    for L, n, par in zip(cache, draft, parents):
        depth = []
        for t in range(n):
            depth.append(1 + (depth[par[t]] if par[t] >= 0 else 0))
        pairs += n * (L - n) + sum(depth)
    return {"bytes": 2 * sum(draft) * H * D * e + 2 * Hkv * D * e * sum(cache), "flops": 4 * D * H * pairs}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    H, Hkv, D = case["H"], case["Hkv"], case["D"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = dict(case=dict(case))
    if case["op"] in ("append", "packed"):
        lens = _lens(case)
        T = sum(lens)
        ends = [sum(lens[:i]) for i in range(len(lens) + 1)]
        # one projection writes q, k and v side by side; the calls take its slices
        qkv = normal(T, H + 2 * Hkv, D)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], cu_seqlens=ints(ends))
        s["longest"] = max(lens)
    if case["op"] == "append":
        s.update(kcache=normal(len(lens), Hkv, case["Skv"], D), vcache=normal(len(lens), Hkv, case["Skv"], D),
                 cache_len=ints([int(case["past"]) + n for n in lens]))
    if case["op"] == "rope":
        s.update(q=normal(case["T"], H, D), k=normal(case["T"], Hkv, D),
                 positions=torch.randint(0, case["far"], (case["T"],), generator=g, device="cuda").to(torch.int32))
    if case["op"] in ("append", "rope"):
        s["freqs"] = torch.tensor(_frequencies(case), dtype=torch.float64)
    if case["op"] == "tree":
        cache, draft, parents = _tree(case)
        B, T = case["B"], case["T"]
        s.update(q=normal(B, T, H, D).transpose(1, 2), kcache=normal(B, Hkv, case["Skv"], D),
                 vcache=normal(B, Hkv, case["Skv"], D), parents=ints(parents), cache_len=ints(cache), draft_len=ints(draft))
    return s


# ------------------------------------------------------------------ plain forms

def _packed_plain(q, k, v, cu, longest, causal):
    T, H, D = q.shape
    Hkv, n = k.shape[1], cu.numel() - 1
    # sequences side by side, padded to the longest
    start, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    at = torch.arange(longest, device=q.device)
    idx = (start[:, None] + at).clamp(max=T - 1)
    inside = at < length[:, None]                                        # (n, longest)
    qp = q.float()[idx].view(n, longest, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, -1, D)
    kp = k.float()[idx].permute(0, 2, 3, 1)                              # (n, Hkv, D, longest)
    vp = v.float()[idx].permute(0, 2, 1, 3)
    s = torch.matmul(qp, kp).view(n, Hkv, H // Hkv, longest, longest)
    s *= 1.0 / math.sqrt(D)
    hidden = ~inside[:, None, :].expand(n, longest, longest)
    if causal:
        hidden = hidden | (at > at[:, None])
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    s -= m
    s.exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(n, Hkv, -1, longest), vp).view(n, Hkv, H // Hkv, longest, D) / l
    lse = (m + l.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, longest, H, D)
    lse = lse.permute(0, 3, 1, 2).reshape(n, longest, H)
    return o[inside].to(q.dtype), lse[inside]


def _rotate_plain(x, positions, freqs, rotary, layout, inverse):
    angle = positions.double()[:, None] * freqs.to(x.device)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    rot, rest = x[..., :rotary], x[..., rotary:]
    if layout == "half":
        a, b = rot[..., :rotary // 2], rot[..., rotary // 2:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((rot, rest), dim=-1)


def _append_plain(s):
    case = s["case"]
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu_seqlens"].long()
    t = torch.arange(q.shape[0], device=q.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    row = s["cache_len"].long()[seq] - (cu[seq + 1] - t)
    args = (row, s["freqs"], case["rotary"], case["layout"], False)
    s["kcache"][seq, :, row] = _rotate_plain(k, *args).to(k.dtype)
    s["vcache"][seq, :, row] = v
    return _rotate_plain(q, *args).to(q.dtype), s["kcache"], s["vcache"]


def _tree_plain(q, kc, vc, parents, cache_len, draft_len):
    B, H, T, D = q.shape
    Hkv, Skv = kc.shape[1], kc.shape[2]
    # ancestors: the parent relation closed by squaring (a token is its own ancestor)
    t = torch.arange(T, device=q.device)
    anc = ((parents[:, :, None] == t) | (t[:, None] == t)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        anc = (torch.matmul(anc, anc) > 0).float()
    past = (cache_len - draft_len).long()
    j = torch.arange(Skv, device=q.device) - past[:, None]                # draft index of each cache row
    drafted = (j >= 0) & (j < draft_len[:, None])
    seen = torch.gather(anc, 2, j.clamp(0, T - 1)[:, None].expand(B, T, Skv)) > 0
    seen = (j < 0)[:, None] | (seen & drafted[:, None])                   # (B, T, Skv)
    qf = q.float().reshape(B, Hkv, H // Hkv * T, D)
    s = torch.matmul(qf, kc.float().transpose(2, 3)).view(B, Hkv, H // Hkv, T, Skv)
    s *= 1.0 / math.sqrt(D)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    s /= s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, -1, Skv), vc.float()).view(B, H, T, D)
    return torch.where((t < draft_len[:, None])[:, None, :, None], o, torch.zeros_like(o)).to(q.dtype)


def run(s):
    case = s["case"]
    if own:
        import transformer_scaled_dot_fwd_gb300 as attn

        if case["op"] == "packed":
            return attn.attn_fwd_packed(s["q"], s["k"], s["v"], s["cu_seqlens"], causal=case["causal"], return_lse=True)
        if case["op"] == "append":
            q = attn.attn_rope_append(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["freqs"],
                                      cu_seqlens=s["cu_seqlens"], cache_len=s["cache_len"],
                                      interleaved=case["layout"] == "interleaved")
            return q, s["kcache"], s["vcache"]
        if case["op"] == "rope":
            return attn.attn_rope(s["q"], s["k"], s["positions"], s["freqs"],
                                  interleaved=case["layout"] == "interleaved", inverse=case["inverse"])
        return attn.attn_decode_tree(s["q"], s["kcache"], s["vcache"], s["parents"], cache_len=s["cache_len"],
                                     draft_len=s["draft_len"])
    if case["op"] == "packed":
        return _packed_plain(s["q"], s["k"], s["v"], s["cu_seqlens"], s["longest"], case["causal"])
    if case["op"] == "append":
        return _append_plain(s)
    if case["op"] == "rope":
        args = (s["positions"], s["freqs"], case["rotary"], case["layout"], case["inverse"])
        return _rotate_plain(s["q"], *args).to(s["q"].dtype), _rotate_plain(s["k"], *args).to(s["k"].dtype)
    return _tree_plain(s["q"], s["kcache"], s["vcache"], s["parents"], s["cache_len"], s["draft_len"])


# ------------------------------------------------------------------ from the definition, in 64 bits

def _attend(q, k, v, visible):
    """softmax(q k^T / sqrt(D)) v of one head over the visible pairs, and the log of the sum."""
    x = (q @ k.T) / math.sqrt(q.shape[-1])
    x = torch.where(visible, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v, lse


def _turned(x, position, case):
    """Every pair of x (T, heads, D) as a complex number, turned by position * frequency."""
    r = case["rotary"]
    x = x.double()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
    else:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2))
    w = torch.tensor(_frequencies(case), dtype=torch.float64, device=x.device)
    angle = position.double()[:, None, None] * w
    z = z * torch.polar(torch.ones_like(angle), -angle if case.get("inverse") else angle)
    out = x.clone()
    if case["layout"] == "half":
        out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
    else:
        out[..., :r] = torch.view_as_real(z).flatten(-2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    H, G = case["H"], case["H"] // case["Hkv"]
    if case["op"] == "rope":
        return _turned(s["q"], s["positions"], case), _turned(s["k"], s["positions"], case)
    if case["op"] == "append":
        q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        kc, vc = s["kcache"].double(), s["vcache"].double()
        first = 0
        for b, n in enumerate(_lens(case)):
            rows, past = slice(first, first + n), int(case["past"])
            position = torch.arange(past, past + n, device="cuda")
            q[rows] = _turned(s["q"][rows], position, case)
            kc[b, :, past:past + n] = _turned(s["k"][rows], position, case).transpose(0, 1)
            vc[b, :, past:past + n] = s["v"][rows].double().transpose(0, 1)
            first += n
        return q, kc, vc
    if case["op"] == "packed":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        first = 0
        for n in _lens(case):
            rows = slice(first, first + n)
            i = torch.arange(n, device="cuda")
            visible = i[:, None] >= i if case["causal"] else torch.ones(n, n, dtype=torch.bool, device="cuda")
            for h in range(H):
                out[rows, h], lse[rows, h] = _attend(s["q"][rows, h].double(), s["k"][rows, h // G].double(),
                                                     s["v"][rows, h // G].double(), visible)
            first += n
        return out, lse
    cache, draft, parents = _tree(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (L, n, par) in enumerate(zip(cache, draft, parents)):
        visible = torch.zeros(n, L, dtype=torch.bool)
        visible[:, :L - n] = True
        for t in range(n):
            j = t
            while j >= 0:
                visible[t, L - n + j] = True
                j = par[j]
        visible = visible.cuda()
        for h in range(H):
            out[b, h, :n] = _attend(s["q"][b, h, :n].double(), s["kcache"][b, h // G, :L].double(),
                                    s["vcache"][b, h // G, :L].double(), visible)[0]
    return out
