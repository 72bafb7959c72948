"""What test_paged_split.py restates of paged attention's division of work is what the
kernel's source says: its constants, and the arithmetic of units, rows and edge tiles, taken
from csrc/paged_tc.cu and compiled for the host.  The host's choice of clusters, grid and
workspace is held to a restatement of its rule, and the clusters' shares to a partition."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
import transformer_scaled_dot_fwd_gb300.build as build
import test_paged_split as split
from test_paged_split import KN, MIN_TILES, UNIT_COST, WEIGHT_TWO, Units, cdiv

TC = open(os.path.join(build.CSRC, "paged_tc.cu")).read()
API = open(os.path.join(build.CSRC, "api.cu")).read()


def constant(name):
    m = re.search(rf"constexpr int {name} = (\d+);", TC)
    assert m, f"no constant {name}"
    return int(m.group(1))


def between(first, last):
    assert TC.count(first) == 1, first
    a = TC.index(first)
    return TC[a:TC.index(last, a)]


def test_constants():
    assert (constant("kN"), constant("kUnitCost"), constant("kMinTiles"), constant("kWeightTwo")) == (KN, UNIT_COST, MIN_TILES, WEIGHT_TWO)
    assert constant("kM") == 128
    # the shortest share of a CTA, as the kernel and as the host count it
    assert "total / (4 * kN * kMinTiles)" in TC and f"axis / {4 * KN * MIN_TILES} < a.n_sm" in API


def test_the_record_names_the_last_share():
    """The restated walk's formula for the CTA in which a unit's last tile begins."""
    assert "const long long last = pos + static_cast<long long>(nt - 1) * units.tile;" in TC
    assert "quotient((last + 1) * N - 1, total)" in TC
    # lo and hi are total I / N and total (I + 1) / N, in parts that stay within 64 bits
    assert "lo = each * I + odd * I / N, hi = each * (I + 1) + odd * (I + 1) / N" in TC
    r = random.Random(3)
    for _ in range(2000):
        total, N = r.randint(1, 1 << r.randint(1, 51)), r.randint(1, 1023)
        each, odd = divmod(total, N)
        I = r.randrange(N)
        assert each * I + odd * I // N == total * I // N and odd * N < 1 << 31


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """The kernel's own functions, compiled for the host."""
    if not shutil.which("g++"):
        pytest.skip("no g++")
    parts = [between("// a / b, in 32 bits", "// A run of K/V tiles"), between("// A run of K/V tiles", "struct GuardReq"),
             between("// First edge tile of a run", "// A cluster's CTA leaves")]
    consts = "\n".join(f"constexpr int {n} = {constant(n)};" for n in ("kN", "kM", "kUnitCost", "kWeightTwo"))
    text = f"""
#include <algorithm>
#define __device__
#define __forceinline__ inline
using std::max; using std::min;
struct PagedArgs {{ int H, H_kv, heads, groups, tokens; }};
struct Seq {{ int c0, n, L; }};
{consts}
{''.join(parts)}
extern "C" {{
long long h_quotient(long long a, long long b) {{ return quotient(a, b); }}
int h_units(int n, int L, int tokens, int one) {{ return Units(Seq{{0, n, L}}, tokens, one).nu; }}
long long h_at(int n, int L, int tokens, int one, int u) {{ return Units(Seq{{0, n, L}}, tokens, one).at(u); }}
int h_cut(int n, int L, int tokens, int one, long long x, int nt) {{ return Units(Seq{{0, n, L}}, tokens, one).cut(x, nt); }}
int h_tiles(int keys) {{ return tiles_of(keys); }}
int h_edge(int tok0, int past, int j0, int n) {{ Run r{{}}; r.tok0 = tok0, r.past = past, r.j0 = j0, r.n = n; return edge_of(r); }}
void h_row(int H, int H_kv, int heads, int groups, int tokens, int hs, int tok0, int left, int past, int x, int r, int *out) {{
    const Row w = row_of(PagedArgs{{H, H_kv, heads, groups, tokens}}, hs, tok0, left, past, x, r);
    out[0] = w.valid, out[1] = w.token, out[2] = w.head, out[3] = w.lim;
}}
}}
"""
    d = tmp_path_factory.mktemp("split")
    src, out = d / "split.cpp", d / "split.so"
    src.write_text(text)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    h = ctypes.CDLL(str(out))
    ll, i = ctypes.c_longlong, ctypes.c_int
    for name, res, args in (("h_quotient", ll, [ll, ll]), ("h_units", i, [i] * 4), ("h_at", ll, [i] * 5), ("h_cut", i, [i] * 4 + [ll, i]),
                            ("h_tiles", i, [i]), ("h_edge", i, [i] * 4)):
        getattr(h, name).restype, getattr(h, name).argtypes = res, args
    return h


def test_units_are_the_restated_ones(host):
    r = random.Random(1)
    for _ in range(4000):
        one = r.choice((1, 2, 16, 25, 32, 64, 128))
        tokens = one * r.choice((1, 2))
        n = r.choice((1, one, one + 1, tokens, tokens + 1, r.randint(1, 5000), r.randint(1, 1 << 22)))
        L = r.choice((0, n // 2, n, n + r.randint(0, 1 << 20), r.randint(0, 0x7fff0000)))
        u = Units(n, L, tokens, one)
        assert host.h_units(n, L, tokens, one) == u.nu
        for i in {0, 1, u.nu // 2, u.nu - 1, u.nu}:
            assert host.h_at(n, L, tokens, one, i) == u.at(i)
        i = r.randrange(u.nu)
        nt = host.h_tiles(u.keys(i))
        assert nt == u.tiles(i)
        for x in (-5, 0, 1, u.tile - 1, u.tile, u.tile + 1, r.randint(0, nt * u.tile), nt * u.tile - 1, nt * u.tile, nt * u.tile + 9):
            assert host.h_cut(n, L, tokens, one, x, nt) == u.cut(x, nt)


def test_quotients(host):
    r = random.Random(2)
    for _ in range(4000):
        a, b = r.randint(0, 1 << r.randint(0, 62)), r.randint(1, 1 << r.randint(0, 62))
        assert host.h_quotient(a, b) == a // b


@pytest.mark.parametrize("G,H_kv", [(1, 2), (3, 2), (4, 8), (5, 1), (33, 2), (128, 1), (130, 2), (300, 1)])
def test_rows_hold_every_token_and_head_once(host, G, H_kv):
    """The rows of a unit's tiles: each (token, head) of its sequence once, with the keys that it sees; tiles in front of
    the edge are seen whole by all of them."""
    groups = cdiv(G, 128)
    heads = cdiv(G, groups)
    tokens = 128 // heads
    out = (ctypes.c_int * 4)()
    r = random.Random(G)
    for n, L in ((1, 1), (tokens, 5 * KN), (2 * tokens + 1, 300), (tokens + 3, 2), (2 * tokens, 0), (r.randint(1, 300), r.randint(0, 2000))):
        seen = set()
        for hs in range(H_kv * groups):
            for tok0 in range(0, n, 2 * tokens):
                lims = []
                for x in range(2):
                    for row in range(128):
                        host.h_row(G * H_kv, H_kv, heads, groups, tokens, hs, tok0, n - tok0, L - n, x, row, out)
                        valid, token, head, lim = out
                        if not valid:
                            continue
                        assert 0 <= token < n and head // G == hs // groups and lim == max(0, L - n + token + 1)
                        assert (token, head) not in seen
                        seen.add((token, head))
                        lims.append(lim)
                nt = host.h_tiles(max(lims)) if lims else 0
                for j0 in {0, nt // 2, max(0, nt - 1)} if lims else ():
                    edge = host.h_edge(tok0, L - n, j0, nt - j0)
                    whole = [all(lim >= (t + 1) * KN for lim in lims) for t in range(j0, nt)]
                    assert edge == (whole.index(False) if False in whole else nt - j0)
        assert len(seen) == n * G * H_kv


@pytest.mark.parametrize("c", [1, 2, 4, 8])
def test_shares_of_a_cluster(c):
    """CTA r of a cluster of c takes tiles [nt r >> s, nt (r + 1) >> s)."""
    assert "j = tiles_of(keys_of(0)) * static_cast<int>(cluster_rank()) >> a.cluster_shift;" in TC
    assert "nt * static_cast<int>(cluster_rank() + 1) >> a.cluster_shift" in TC
    s = c.bit_length() - 1
    for nt in range(1, 300):
        tiles = [t for r in range(c) for t in range(nt * r >> s, nt * (r + 1) >> s)]
        assert tiles == list(range(nt))


def sizes(T, n_seq, H, H_kv, D, max_len, ragged, n_sm):
    """(CTAs of a cluster or 0, bytes of workspace) of a bf16 call, by the host's rule."""
    G = H // H_kv
    groups = cdiv(G, 128)
    heads = cdiv(G, groups)
    tokens = 128 // heads
    most = T if ragged else T // n_seq
    single, box_tokens = most <= tokens, min(most, tokens)
    slot_rows = cdiv(box_tokens * heads, 32) * 32 if single else 256
    units = n_seq * H_kv * groups
    cluster = next((c for c in (8, 4, 2, 1) if single and 3 * units * c <= (3 if c < 4 else 2) * n_sm), 0)
    if cluster:
        shared = units * (n_seq + 1.0) / (2.0 * n_seq) / n_sm
        if max_len / 128.0 * (1.0 / cluster - shared) > 6.0:
            cluster = 0
    if cluster:
        return cluster, 0
    axis = (n_seq + T / tokens) * H_kv * groups * (WEIGHT_TWO * (float(max_len) + T + KN) + 4 * KN * UNIT_COST)
    grid = min(int(axis / (4 * KN * MIN_TILES)) + 1 if axis / (4 * KN * MIN_TILES) < n_sm else n_sm, 1023)
    return 0, grid * 32 + 2 * grid * slot_rows * (D + 2) * 4


def test_clusters_grid_and_workspace_of_a_call(attn_lib):
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    r = random.Random(6)
    forms = set()
    for _ in range(3000):
        H_kv = r.choice((1, 2, 8, 32))
        H, D, P = H_kv * r.choice((1, 3, 4, 16, 40, 130)), r.choice((64, 128)), r.choice((8, 16, 24, 64))
        n_seq, ragged = r.choice((1, 2, 4, 9, 16, 40, 300)), r.choice((0, 1))
        T = r.choice((1, 7, 40, 3000)) if ragged else n_seq * r.choice((1, 1, 1, 3, 200))
        M = r.choice((0, 1, 9, 90, 900, 9000))
        cluster, need = sizes(T, n_seq, H, H_kv, D, M * P, ragged, n_sm)
        forms.add(cluster)
        assert attn_lib.attn_fwd_paged_workspace(T, n_seq, H, H_kv, D, M, P, ragged, attn.ATTN_BF16) == need
    assert forms == {0, 1, 2, 4, 8}


@pytest.mark.parametrize("seed", range(20))
def test_the_grid_holds_every_share(seed):
    """The axis of any valid offsets is within the host's bound, so that no share is missing; with few units a share has as
    many tiles as the kernel asks for."""
    r = random.Random(seed)
    tokens = r.choice((1, 8, 32, 64))
    per = r.choice((1, 8))
    max_len = r.choice((0, 100, 3000))
    seqs = [(n, r.randint(0, max_len)) for n in (r.choice((0, 1, 1, tokens, r.randint(1, 500))) for _ in range(r.choice((1, 4, 30))))]
    T = sum(n for n, _ in seqs)
    total = sum(Units(n, L, 2 * tokens, tokens).at(cdiv(n, 2 * tokens)) * per for n, L in seqs if n)
    axis = (len(seqs) + T / tokens) * per * (WEIGHT_TWO * (max_len + T + KN) + 4 * KN * UNIT_COST)
    assert total <= axis
    grid = int(axis / (4 * KN * MIN_TILES)) + 1
    assert max(1, total // (4 * KN * MIN_TILES)) <= grid
    N = split.runs_of(seqs, per, 2 * tokens, tokens, min(grid, 152), 0)[2]
    assert N == max(1, min(total // (4 * KN * MIN_TILES), grid, 152))
