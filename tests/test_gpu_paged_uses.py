"""Uses of a paged cache that its contract allows: expanded and sliced pools, expanded
tables, one pool for keys and values, contiguous caches as pages, calls on several streams
at once, captured calls that share one memory pool.  Each is held to the same call on plain
contiguous tensors, whose results other tests hold to the definition: the same bits."""
from __future__ import annotations

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from test_gpu_paged import BF16, F32, SEQS, Paged, ints

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("seqs", [SEQS, [(13, 1)], [(16, 5)]])
def test_one_head_expanded(gpu, seqs, dtype, D):
    """Head stride 0: every cached head is the same rows; pools of many pages and of one."""
    x = Paged(seqs, 8, 1, D, 16, dtype, seed=2, junk=0.0)
    one = len(seqs) == 1
    kp, vp = (t[int(x.table[0, 0]):][:1] if one else t for t in (x.kp, x.vp))
    table = torch.zeros_like(x.table) if one else x.table
    for H_kv in (2, 8):
        a = attn.attn_fwd_paged(x.q, *(t.expand(-1, H_kv, -1, -1) for t in (kp, vp)), table, x.lens, x.cu, return_lse=True)
        b = attn.attn_fwd_paged(x.q, *(t.repeat(1, H_kv, 1, 1) for t in (kp, vp)), table, x.lens, x.cu, return_lse=True)
        attn.attn_device_status()
        assert same(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pools_sliced_by_head_and_column(gpu, dtype):
    """Some heads of wider pools, and keys and values side by side in the rows of one."""
    x = Paged(SEQS, 4, 2, 64, 16, dtype, seed=3)
    want = x.call(return_lse=True)
    wide = [torch.full((x.n_pages, 5, 16, 64), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    for w, t in zip(wide, (x.kp, x.vp)):
        w[:, 2:4] = t
    both = torch.cat((x.kp, x.vp), -1)
    rows = both.transpose(1, 2).contiguous().transpose(1, 2)  # (n_pages, page_size, H_kv, 2 D)
    for k, v in ((wide[0][:, 2:4], wide[1][:, 2:4]), (both[..., :64], both[..., 64:]), (rows[..., :64], rows[..., 64:])):
        x.kp, x.vp = k, v
        assert same(x.call(return_lse=True), want)
    attn.attn_device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_pool_for_keys_and_values(gpu, dtype):
    x = Paged(SEQS, 4, 2, 64, 16, dtype, seed=4)
    a = attn.attn_fwd_paged(x.q, x.kp, x.kp, x.table, x.lens, x.cu, return_lse=True)
    b = attn.attn_fwd_paged(x.q, x.kp, x.kp.clone(), x.table, x.lens, x.cu, return_lse=True)
    attn.attn_device_status()
    assert same(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_row_of_the_table_for_all(gpu, dtype):
    """A table expanded over its sequences, of different lengths."""
    x = Paged([(300, 20)], 4, 2, 64, 16, dtype, seed=5)
    q = torch.randn(7, 4, 64, device="cuda").to(dtype)
    table = x.table[:1].expand(7, -1)
    lens = ints([300, 1, 0, 17, 299, 128, 16])
    a = attn.attn_fwd_paged(q, x.kp, x.vp, table, lens, return_lse=True)
    b = attn.attn_fwd_paged(q, x.kp, x.vp, table.contiguous(), lens, return_lse=True)
    attn.attn_device_status()
    assert same(a, b) and bool((a[1][2] == -torch.inf).all())
    lens = ints([64] * 7)
    assert all(same([s], [t]) for s, t in zip(attn.attn_pages_step(table, lens, x.n_pages, 16), attn.attn_pages_step(table.contiguous(), lens, x.n_pages, 16)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Skv", [8, 264, 1024])
def test_contiguous_caches_as_pages(gpu, Skv, dtype):
    """One page a sequence, its rows no power of two."""
    seqs = [(Skv, 3), (1, 1), (Skv - 5, 1), (Skv // 2, 3), (0, 0)]
    x = Paged(seqs, 6, 3, 64, Skv, dtype, seed=6)
    out, lse = x.call(return_lse=True)
    attn.attn_device_status()
    x.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_append_to_rows_that_hold_both(gpu, D):
    """Keys and values side by side in the rows of one pool; copies in it."""
    g = torch.Generator().manual_seed(7)
    freqs = attn.attn_rope_frequencies(D)
    q, k, v = (torch.randn(5, h, D, generator=g).to(BF16).cuda() for h in (4, 2, 2))
    table, lens, cu = ints([[3, 1], [0, 2]]), ints([18, 2]), ints([0, 3, 5])
    both = torch.zeros(4, 2, 16, 2 * D, dtype=BF16, device="cuda")
    apart = [torch.zeros(4, 2, 16, D, dtype=BF16, device="cuda") for _ in range(2)]
    a = attn.attn_rope_append_paged(q, k, v, both[..., :D], both[..., D:], table, freqs, lens, cu)
    b = attn.attn_rope_append_paged(q, k, v, *apart, table, freqs, lens, cu)
    c = ints([[1, 0, 16], [-1, -1, 0], [3, 2, 9]])
    attn.attn_pages_copy(both[..., :D], both[..., D:], c)
    attn.attn_pages_copy(*apart, c)
    assert torch.equal(a, b) and torch.equal(both, torch.cat(apart, -1)) and torch.count_nonzero(both[0])


def test_clusters_on_several_streams_at_once(gpu):
    """Small calls whose kernels are clusters, bf16 and fp32, with steps of a table beside them."""
    xs = [Paged([(700 + 90 * i, 1)] * n, 8, 2, D, 16, dtype, seed=40 + i, even=True)
          for i, (n, D, dtype) in enumerate([(1, 64, BF16), (1, 128, BF16), (3, 64, BF16), (2, 64, F32), (1, 128, F32)])]
    want = [x.call() for x in xs]
    tables = [attn.attn_pages_step(x.table, x.lens, x.n_pages, 16, new_len=x.lens + 1) for x in xs]
    moved = [attn.attn_pages_compact(x.table, x.lens, x.n_pages, 16) for x in xs]
    new = [x.lens + 1 for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for r in range(30):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got.append((i, x.call(), attn.attn_pages_step(x.table, x.lens, x.n_pages, 16, new_len=new[i]),
                            attn.attn_pages_compact(x.table, x.lens, x.n_pages, 16)))
    torch.cuda.synchronize()
    attn.attn_device_status()
    for i, out, step, compact in got:
        assert torch.equal(out, want[i]) and same(step, tables[i]) and same(compact, moved[i])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_graphs_of_one_memory_pool(gpu, dtype):
    """Captured calls with workspaces, replayed in turn: what one leaves in shared memory of the pool is nothing to the other."""
    xs = [Paged([(2500, 130), (900, 1), (1800, 40)], 8, 2, 64, 16, dtype, seed=50), Paged([(6000, 1)] * 3, 8, 2, 64, 16, dtype, seed=51, even=True)]
    want = [x.call(return_lse=True) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pool, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool, stream=side):
            outs.append(x.call(return_lse=True))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same(outs[i], want[i])
    attn.attn_device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_that_decrease_stay_inside(gpu, dtype):
    """Offsets that are none: the rows of sequences that overlap are undefined, everything around the tensors stays."""
    x = Paged([(300, 60), (200, 40), (500, 1), (64, 64)], 4, 2, 64, 16, dtype, seed=8)
    room = torch.full((x.T + 64, 4, 64), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((x.T + 64, 4), 5.0, device="cuda")
    for cu in ([0, 165, 3, 165, 165], [165, 0, 165, 0, 165], [-9, 70, 20, 1 << 30, 40], [7, 7, 7, 7, 7], [-(1 << 31), (1 << 31) - 1, 0, 0, 0]):
        x.cu = ints(cu)
        x.call(out=room[32:-32], lse=lse[32:-32])
        torch.cuda.synchronize()
        attn.attn_device_status()
        for t in (room, lse):
            assert bool((t[:32] == 5).all()) and bool((t[-32:] == 5).all())
