"""GPU parity tests of attn_fwd_packed against the definition in 64 bits, sequence
by sequence; the tolerances are derived in serving_ref.py."""
from __future__ import annotations

import math

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import workloads as wl
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(lens, lead=0):
    return [lead + sum(lens[:i]) for i in range(len(lens) + 1)]


def tokens(T, H, H_kv, D, seed, dtype):
    """q, k, v as slices of one fused projection."""
    x = wl.random_tensors((max(T, 1), H + 2 * H_kv, D), seed, dtype=dtype, count=1)[0][:T]
    return x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]


def verify(q, k, v, cu, causal, out, lse, scale=None, what="", only=None):
    T, H, D = q.shape
    G = H // k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            continue
        i = torch.arange(b - a, device="cuda")
        visible = i[:, None] >= i if causal else torch.ones(b - a, b - a, dtype=torch.bool, device="cuda")
        for h in range(H) if only is None else only:
            o, l, A, size = ref.attend(q[a:b, h], k[a:b, h // G], v[a:b, h // G], visible, scale)
            tol, ltol = ref.bounds(q.dtype, D, b - a, scale, size, o, A)
            ref.check(out[a:b, h], o, tol, f"{what} sequence {s} ({b - a} tokens) head {h}")
            if lse is not None:
                err = (lse[a:b, h].double() - l).abs()
                assert torch.all(err <= ltol + l.abs() * 2.0 ** -22), f"{what} lse {s} {h}: {err.max():.3e}"


def case(lens, H, H_kv, D, causal, dtype=BF16, seed=1, scale=None, lead=0, trail=0, only=None):
    T = sum(lens) + lead + trail
    q, k, v = tokens(T, H, H_kv, D, seed, dtype)
    cu = offsets(lens, lead)
    out = torch.full((T, H, D), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((T, H), 5.0, dtype=F32, device="cuda")
    got = attn.attn_fwd_packed(q, k, v, ints(cu), out=out, lse=lse, causal=causal, scale=scale)
    attn.attn_device_status()
    assert got[0] is out and got[1] is lse
    verify(q, k, v, cu, causal, out, lse, scale, f"lens {lens[:6]} H {H}/{H_kv} D {D} causal {causal}", only)
    for x in (out, lse):  # rows outside every sequence stay as they were
        assert torch.all(x[:lead] == 5.0) and torch.all(x[T - trail:] == 5.0)
    return q, k, v, cu, out, lse


LENS = [[1], [5, 0, 1, 127, 128, 129], [64, 300, 2], [257, 512, 33, 0], [0, 0, 1000, 0], [1] * 40]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,H_kv", [(4, 4), (4, 2), (6, 2), (8, 1), (1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_packed_bf16(gpu, lens, H, H_kv, D, causal):
    case(lens, H, H_kv, D, causal, seed=len(lens), lead=3, trail=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,H_kv", [(2, 2), (6, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_packed_fp32(gpu, lens, H, H_kv, D, causal):
    case(lens, H, H_kv, D, causal, dtype=F32, seed=len(lens), lead=3, trail=2)


def test_long_sequences(gpu):
    case([3001, 1, 4100, 700], 8, 2, 128, True, seed=3, only=(0, 7))
    case([2999], 2, 1, 64, False, dtype=F32, seed=4)


def test_many_sequences(gpu):
    """More sequences than the plan kernel has threads."""
    case([(5 * i) % 7 for i in range(2500)], 2, 1, 64, True, seed=5, only=(1,))
    case([(5 * i) % 7 for i in range(1300)], 1, 1, 64, True, dtype=F32, seed=5)


def test_a_sequence_past_the_plan_s_index_range(gpu):
    """More than 1024 query tiles in one sequence: they share the last place of
    the plan's order.  Checked on the first, some middle and the last rows."""
    T, D = 150000, 64
    q, k, v = tokens(T + 50, 2, 1, D, 6, BF16)
    out, lse = attn.attn_fwd_packed(q, k, v, ints([0, T, T + 50]), causal=True, return_lse=True)
    attn.attn_device_status()
    for a in (0, 131000, 131072, T - 70):
        i = torch.arange(a, a + 64, device="cuda")
        visible = i[:, None] >= torch.arange(T, device="cuda")
        for h in (0, 1):
            o, l, A, size = ref.attend(q[a:a + 64, h], k[:T, 0], v[:T, 0], visible, D ** -0.5)
            tol, ltol = ref.bounds(BF16, D, T, D ** -0.5, size, o, A)
            ref.check(out[a:a + 64, h], o, tol, f"row {a}")
            assert torch.all((lse[a:a + 64, h].double() - l).abs() <= ltol + l.abs() * 2.0 ** -22)
    verify(q[T:], k[T:], v[T:], [0, 50], True, out[T:], lse[T:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales(gpu, dtype):
    for scale in (0.0, 1.0, 1e-3):
        case([70, 130], 4, 2, 64, True, dtype=dtype, scale=scale, seed=7)
        case([70, 130], 4, 2, 64, False, dtype=dtype, scale=scale, seed=7)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_masked_infinities_leave_no_trace(gpu, dtype, causal, D):
    """Infinities and NaN in other sequences' K and V, in tokens of no sequence,
    and (causal) in later tokens of the same sequence: the rows that do not see
    them equal, bit for bit, the rows computed without them."""
    lens, lead, trail = [100, 0, 200, 131, 60], 5, 70
    T = sum(lens) + lead + trail
    cu = offsets(lens, lead)
    q, k, v = (x.contiguous() for x in tokens(T, 4, 2, D, 8, dtype))
    clean = attn.attn_fwd_packed(q, k, v, ints(cu), causal=causal, return_lse=True)
    k2, v2 = k.clone(), v.clone()
    bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda").to(dtype)
    for x in (k2, v2):
        x[:lead], x[cu[-1]:] = bad[0], bad[1]
        x[cu[2]:cu[3], 1, ::3] = bad[2]           # the whole third sequence, head 1
        x[cu[3] + 77, 0, 5] = bad[0]               # one element of one token of the fourth
    dirty = attn.attn_fwd_packed(q, k2, v2, ints(cu), causal=causal, return_lse=True)
    attn.attn_device_status()
    same = torch.zeros(T, 4, dtype=torch.bool)
    same[cu[0]:cu[1]] = same[cu[4]:cu[5]] = True
    same[cu[2]:cu[3], :2] = True                   # heads 0 and 1 read kv head 0
    same[cu[3]:cu[4], 2:] = True
    if causal:
        same[cu[3]:cu[3] + 77, :2] = True
    for a, b in zip(clean, dirty):
        assert torch.equal(a[same.cuda()], b[same.cuda()])
    # rows that do see the NaN key carry it
    assert torch.isnan(dirty[0][cu[3] + 77, 0]).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_visible_infinities_are_kept(gpu, dtype, causal):
    """An infinite value (finite keys) is infinite in exactly the rows and
    columns that see it, with its sign; two of opposite sign make a NaN."""
    lens = [300, 90]
    q, k, v = (x.contiguous() for x in tokens(390, 2, 1, 128, 9, dtype))
    v[250, 0, 7], v[260, 0, 7], v[310, 0, 100], v[20, 0, 0] = math.inf, -math.inf, -math.inf, math.inf
    out = attn.attn_fwd_packed(q, k, v, ints([0, 300, 390]), causal=causal)
    attn.attn_device_status()
    for h in range(2):
        for a, b in ((0, 300), (300, 390)):
            i = torch.arange(b - a, device="cuda")
            visible = i[:, None] >= i if causal else torch.ones(b - a, b - a, dtype=torch.bool, device="cuda")
            pos = (visible.double() @ (v[a:b, 0] == math.inf).double()) > 0
            neg = (visible.double() @ (v[a:b, 0] == -math.inf).double()) > 0
            got = out[a:b, h].float()
            assert torch.equal(torch.isnan(got), pos & neg)
            assert torch.equal(got == math.inf, pos & ~neg) and torch.equal(got == -math.inf, neg & ~pos)


@pytest.mark.parametrize("part", [1.0, 0.5])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_at_the_type_s_limits(gpu, dtype, part):
    """Scores near the type's lowest finite value are scores, not masks, as far as
    their base-2 exponent (1.44 times the score) is an fp32 number: half the
    lowest value is, the lowest value itself counts as -inf, and a row of
    nothing else is a NaN."""
    q, k, v = (x.contiguous() for x in tokens(200, 2, 1, 64, 10, dtype))
    k[50:120] *= 0
    q[:, :, 1:], k[:, :, 1:] = 0, 0
    q[:, :, 0] = 1
    k[:, 0, 0] = -part * torch.finfo(torch.bfloat16).max   # every score the same, about -3e38
    out = attn.attn_fwd_packed(q, k, v, ints([0, 200]), scale=1.0, causal=True)
    attn.attn_device_status()
    if part == 1.0:
        assert torch.isnan(out).all()
        return
    mean = v[:, 0].double().cumsum(0) / torch.arange(1, 201, device="cuda")[:, None]
    size = v[:, 0].double().abs().cumsum(0) / torch.arange(1, 201, device="cuda")[:, None]
    tol = size * (torch.finfo(dtype).eps + 2.0 ** -14)
    for h in range(2):
        ref.check(out[:, h], mean, tol)


def test_strided_layouts_agree(gpu):
    """Contiguous tensors, fused slices and head-major views give the same bits."""
    lens, H, H_kv, D = [130, 40, 77], 4, 2, 128
    q, k, v = tokens(247, H, H_kv, D, 11, BF16)
    cu = ints(offsets(lens))
    a = attn.attn_fwd_packed(q, k, v, cu, causal=True)
    b = attn.attn_fwd_packed(q.contiguous(), k.contiguous(), v.contiguous(), cu, causal=True)
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    o = torch.empty((H, 247, D), dtype=BF16, device="cuda").transpose(0, 1)
    c = attn.attn_fwd_packed(*hm, cu, out=o, causal=True)
    wide = torch.zeros(247, H + 3, D, dtype=BF16, device="cuda")
    d = attn.attn_fwd_packed(q, k, v, cu, out=wide[:, 2:2 + H], causal=True)
    attn.attn_device_status()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    assert torch.count_nonzero(wide[:, :2]) == 0 and torch.count_nonzero(wide[:, 2 + H:]) == 0


def test_one_sequence_equals_dense_prefill(gpu):
    """The same tiles in the same order: bit for bit attn_fwd of that sequence."""
    S, H, H_kv, D = 700, 8, 2, 128
    q, k, v = (x.contiguous() for x in tokens(S, H, H_kv, D, 12, BF16))
    dense = [x.transpose(0, 1)[None].contiguous() for x in (q, k, v)]
    for causal in (True, False):
        out = attn.attn_fwd_packed(q, k, v, ints([0, S]), causal=causal)
        want = attn.attn_fwd(*dense, causal=causal)
        attn.attn_device_status()
        assert torch.equal(out, want[0].transpose(0, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_malformed_offsets_stay_inside(gpu, dtype):
    """Decreasing or out-of-range offsets: no access outside the tensors, the
    device status stays clean, and the next call is right."""
    q, k, v = tokens(300, 4, 2, 64, 13, dtype)
    guard = torch.full((300 + 64, 4, 64), 3.0, dtype=dtype, device="cuda")
    for cu in ([0, 400, 200, 300], [-9, 5, 2000000000, 300], [300, 200, 100, 0], [7, 7, 7, 7], [-5, -4, -3, -2],
               [0, 300, 0, 300], [0, 300, 0, 300, 0, 300, 0, 300]):
        attn.attn_fwd_packed(q, k, v, ints(cu), out=guard[32:332], causal=True)
        attn.attn_device_status()
    assert torch.all(guard[:32] == 3.0) and torch.all(guard[332:] == 3.0)
    case([100, 200], 4, 2, 64, True, dtype=dtype, seed=13)


def test_offsets_past_32_bits(gpu):
    """Token rows whose element offset passes 2^31 (and bytes 2^32)."""
    T, H, D = 140000, 132, 128   # 2.37e9 elements
    q = torch.zeros((T, H, D), dtype=BF16, device="cuda")
    k, v = wl.random_tensors((T, 1, D), 14, count=2)
    q[-60:] = wl.random_tensors((60, H, D), 15, count=1)[0]
    out = torch.empty_like(q)
    lens = [T - 60 - 400, 400, 60]
    cu = offsets([1] * 8 + [lens[0] - 8 - 139000] + [139000 // 139] * 139 + lens[1:])
    lse = attn.attn_fwd_packed(q, k, v, ints(cu), out=out, causal=True, return_lse=True)[1]
    attn.attn_device_status()
    verify(q[-60:], k[-60:], v[-60:], [0, 60], True, out[-60:], lse[-60:], only=(0, 77, 131))


def test_streams_graphs_and_two_calls_at_once(gpu):
    lens = [400, 33, 0, 129]
    T, H, H_kv, D = sum(lens), 4, 2, 128
    cu = ints(offsets(lens))
    q, k, v = tokens(T, H, H_kv, D, 16, BF16)
    q2, k2, v2 = tokens(T, H, H_kv, D, 17, BF16)
    cu2 = ints(offsets([50, 200, 300, T - 550]))
    want, want2 = attn.attn_fwd_packed(q, k, v, cu, causal=True), attn.attn_fwd_packed(q2, k2, v2, cu2, causal=True)
    torch.cuda.synchronize()
    # two streams at once: each call has a plan of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((attn.attn_fwd_packed(q, k, v, cu, causal=True, stream=s1), want))
        outs.append((attn.attn_fwd_packed(q2, k2, v2, cu2, causal=True, stream=s2.cuda_stream), want2))
    torch.cuda.synchronize()
    attn.attn_device_status()
    for got, w in outs:
        assert torch.equal(got, w)
    # two graphs captured one after the other, replayed side by side, with new lengths
    out, out2 = torch.empty_like(want), torch.empty_like(want2)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.attn_fwd_packed(q, k, v, cu, out=out, causal=True)
    with torch.cuda.graph(g2):
        attn.attn_fwd_packed(q2, k2, v2, cu2, out=out2, causal=True)
    for _ in range(5):
        with torch.cuda.stream(s1):
            g.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out2, want2)
    cu.copy_(ints(offsets([100, 100, 100, T - 300])))
    g.replay()
    torch.cuda.synchronize()
    attn.attn_device_status()
    assert torch.equal(out, attn.attn_fwd_packed(q, k, v, cu, causal=True))


def test_repeated_calls_give_the_same_bits(gpu):
    q, k, v = tokens(3000, 8, 2, 64, 18, BF16)
    cu = ints(offsets([1000, 7, 993, 500, 500]))
    first = attn.attn_fwd_packed(q, k, v, cu, causal=True, return_lse=True)
    for _ in range(10):
        again = attn.attn_fwd_packed(q, k, v, cu, causal=True, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_empty_calls_and_refusals(gpu):
    q, k, v = (x.contiguous() for x in tokens(8, 4, 2, 64, 19, BF16))
    cu = ints([0, 8])
    assert attn.attn_fwd_packed(q[:0], k[:0], v[:0], ints([0, 0])).shape == (0, 4, 64)
    out = torch.full_like(q, 2.0)
    attn.attn_fwd_packed(q, k, v, ints([0]), out=out)  # no sequence
    assert torch.all(out == 2.0)
    for args in ((q, k[:7], v, cu), (q, k, v[:, :1], cu), (q, k, v, cu.long()), (q, k, v, None), (q, k, v, cu.cpu()),
                 (q, torch.cat([k, k[:, :1]], 1), torch.cat([v, v[:, :1]], 1), cu), (q.transpose(1, 2), k, v, cu)):
        with pytest.raises((ValueError, AttributeError)):
            attn.attn_fwd_packed(*args)
    with pytest.raises(TypeError):
        attn.attn_fwd_packed(q.half(), k.half(), v.half(), cu)
    with pytest.raises(TypeError):
        attn.attn_fwd_packed(q, k.float(), v, cu)
    for kw in (dict(out=q), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(attn.AttnError) as e:
            attn.attn_fwd_packed(q, k, v, cu, **kw)
        assert e.value.code == attn.ATTN_EINVAL
    odd = torch.zeros(8, 4, 68, dtype=BF16, device="cuda")[..., :64]  # rows 136 bytes apart
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_packed(odd, k, v, cu)
    with pytest.raises(attn.AttnError) as e:
        x = torch.zeros(8, 2, 96, dtype=BF16, device="cuda")
        attn.attn_fwd_packed(x, x.clone(), x.clone(), cu)
    assert e.value.code == attn.ATTN_EUNSUPPORTED


# Few sequences: each CTA makes the plan; many, or many tiles: the plan kernel.  What
# a row computes does not depend on where its tile stands in the plan.
@pytest.mark.parametrize("H,H_kv", [(2, 1), (3, 3)])
@pytest.mark.parametrize("lens", [[300, 1, 0, 128, 129, 700], [37] * 32, [257] * 31 + [1], [0] * 31 + [900]])
@pytest.mark.parametrize("causal", [True, False])
def test_both_plans_give_the_same_bits(gpu, lens, H, H_kv, causal):
    q, k, v = tokens(sum(lens), H, H_kv, 64, 12, BF16)
    few = attn.attn_fwd_packed(q, k, v, ints(offsets(lens)), causal=causal, return_lse=True)
    many = attn.attn_fwd_packed(q, k, v, ints(offsets([0] * 20 + lens + [0] * 20)), causal=causal, return_lse=True)
    attn.attn_device_status()
    assert torch.equal(few[0], many[0]) and torch.equal(few[1], many[1])


# T / 128 + n_seq = 384 is the last that fits the CTAs' own plan
@pytest.mark.parametrize("T", [383 * 128 - 1, 383 * 128, 383 * 128 + 127, 384 * 128])
def test_plans_at_the_most_tiles(gpu, T):
    q, k, v = tokens(T, 2, 1, 64, 13, BF16)
    lse = torch.full((T, 2), 5.0, device="cuda")
    out, _ = attn.attn_fwd_packed(q, k, v, ints([0, T]), lse=lse, causal=True)
    want, wl_ = attn.attn_fwd_packed(q, k, v, ints([0, T] + [T] * 40), causal=True, return_lse=True)
    attn.attn_device_status()
    assert torch.equal(out, want) and torch.equal(lse, wl_)


@pytest.mark.parametrize("n", [16, 40])
def test_overlapping_sequences_stay_inside(gpu, n):
    # every other sequence holds all tokens: more tile units than the plan has places
    T = 4000
    q, k, v = tokens(T, 2, 1, 64, 14, BF16)
    big = torch.full((T + 2, 2, 64), 5.0, dtype=BF16, device="cuda")
    attn.attn_fwd_packed(q, k, v, ints([0, T] * n), out=big[1:T + 1], causal=True)
    attn.attn_device_status()
    assert torch.all(big[0] == 5) and torch.all(big[-1] == 5)


# fp32: few blocks are clusters of 2, 4 or 8 CTAs that share the keys
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[200], [300, 200], [600], [1100], [1025, 1]])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_clusters(gpu, lens, D, causal):
    case(lens, 2, 1, D, causal, dtype=F32, seed=21)


# fp32: many short blocks take half the workers, two blocks an SM
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[50] * 90, [200, 1, 129] * 20])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_many_blocks(gpu, lens, D, causal):
    case(lens, 4, 2, D, causal, dtype=F32, seed=22)


@pytest.mark.parametrize("H,H_kv", [(4, 2), (3, 3)])
def test_bf16_rows_do_not_depend_on_the_batch(gpu, H, H_kv):
    lens = [300, 1, 129, 0, 700, 64]
    q, k, v = tokens(sum(lens), H, H_kv, 128, 23, BF16)
    cu = offsets(lens)
    out, lse = attn.attn_fwd_packed(q, k, v, ints(cu), causal=True, return_lse=True)
    for a, b in zip(cu, cu[1:]):
        if a < b:
            alone = attn.attn_fwd_packed(q[a:b], k[a:b], v[a:b], ints([0, b - a]), causal=True, return_lse=True)
            assert torch.equal(alone[0], out[a:b]) and torch.equal(alone[1], lse[a:b])
    attn.attn_device_status()


@pytest.mark.parametrize("lens", [[300, 200], [700, 513, 260, 129, 64, 1], [60] * 80])
def test_fp32_repeated_calls_give_the_same_bits(gpu, lens):
    q, k, v = tokens(sum(lens), 4, 4, 64, 24, F32)
    first = attn.attn_fwd_packed(q, k, v, ints(offsets(lens)), return_lse=True)
    for _ in range(5):
        again = attn.attn_fwd_packed(q, k, v, ints(offsets(lens)), return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_a_seen_infinity_is_never_lost(gpu, dtype, causal, D):
    """A key whose weight underflows (its score lies some 1400 below the others)
    with an infinite or NaN value: the element is infinite or NaN in every row that
    sees the key, whichever keys the row's neighbours see, and in no other."""
    lens = [300, 45]
    q, k, v = (x.contiguous() for x in tokens(345, 2, 1, D, 31, dtype))
    q[..., 0] = 8.0
    for row, col, x in ((17, 3, math.inf), (70, 20, -math.inf), (295, 41, math.nan), (305, 5, math.inf)):
        k[row, 0, 0] = -180.0 * math.sqrt(D)
        v[row, 0, col] = x
    out = attn.attn_fwd_packed(q, k, v, ints([0, 300, 345]), causal=causal)
    attn.attn_device_status()
    for a, b in ((0, 300), (300, 345)):
        i = torch.arange(b - a, device="cuda")
        visible = i[:, None] >= i if causal else torch.ones(b - a, b - a, dtype=torch.bool, device="cuda")
        hit = (visible.double() @ (~torch.isfinite(v[a:b, 0])).double()) > 0
        for h in range(2):
            assert torch.equal(~torch.isfinite(out[a:b, h]), hit)
            o, _, A, size = ref.attend(q[a:b, h], k[a:b, 0], v[a:b, 0], visible, D ** -0.5)
            tol, _ = ref.bounds(dtype, D, b - a, D ** -0.5, size, o, A)
            got = torch.where(hit, torch.zeros_like(o), out[a:b, h].double())
            ref.check(got, torch.where(hit, torch.zeros_like(o), o), tol)



@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_rows_of_infinitely_low_scores(gpu, dtype, n):
    """A row whose every score is -inf is a NaN with a log-sum-exp of -inf; keys of
    such scores beside an ordinary one have no weight."""
    q, k, v = (x.contiguous() for x in tokens(2 * n, 2, 1, 64, 38, dtype))
    q[..., 3] = 2.0
    k[:n, 0, 3] = -math.inf
    k[n:2 * n - 1, 0, 3] = -math.inf
    out, lse = attn.attn_fwd_packed(q, k, v, ints([0, n, 2 * n]), return_lse=True)
    attn.attn_device_status()
    assert torch.isnan(out[:n]).all() and torch.all(lse[:n] == -math.inf)
    assert torch.equal(out[n:], v[2 * n - 1:].expand(n, 2, 64))
    s = (q[n:].double() @ k[-1, 0].double()) / 8
    assert torch.all((lse[n:].double() - s).abs() <= 70 * 2.0 ** -23 * 16 + s.abs() * 2.0 ** -22)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,H_kv,D", [(2, 1, 128), (2, 2, 64)])
def test_huge_scores_stay_in_their_rows(gpu, dtype, causal, H, H_kv, D):
    """Scores of huge or infinite magnitude in the next sequence, in tokens of no
    sequence and in other rows of the same sequence: the rows that have no part in
    them keep their bits, out and lse."""
    lens, trail = [100, 75, 60], 40
    T = sum(lens) + trail
    cu = offsets(lens)
    q, k, v = (x.contiguous() for x in tokens(T, H, H_kv, D, 32, dtype))
    clean = attn.attn_fwd_packed(q, k, v, ints(cu), causal=causal, return_lse=True)
    at = torch.arange(T, device="cuda")

    def check(q, k, keep, what):
        got = attn.attn_fwd_packed(q, k, v, ints(cu), causal=causal, return_lse=True)
        attn.attn_device_status()
        for a, b in zip(clean, got):
            assert torch.equal(a[keep], b[keep]), what

    q2 = q.clone()
    q2[cu[1]:cu[2]] *= 1e9
    q2[cu[3]:] *= -1e9
    check(q2, k, (at < cu[1]) | ((at >= cu[2]) & (at < cu[3])), "the next sequence's q")
    for x in (1e9, math.inf):
        q2 = q.clone()
        q2[20, :, 3] = x          # a row in the midst of a warp's
        q2[cu[2] + 59] *= 1e12    # and the last of a sequence
        check(q2, k, (at < cu[3]) & (at != 20) & (at != cu[2] + 59), "one row's q")
    if causal:
        for x in (1e9, math.inf, -math.inf):
            k2 = k.clone()
            k2[20, :, 3] = x
            k2[cu[1] + 50, :, 0] = x
            check(q, k2, (at < 20) | ((at >= cu[1]) & (at < cu[1] + 50)) | ((at >= cu[2]) & (at < cu[3])), "a later key")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,H_kv,D", [(2, 1, 128), (2, 2, 64)])
def test_distinct_scores_of_huge_magnitude(gpu, dtype, causal, H, H_kv, D):
    """Scores of 2^27 to 2^92 of both signs, growing over the tiles, beside rows of zeros."""
    cu = offsets([700, 130, 33])
    T = cu[-1]
    v = wl.random_tensors((T, H_kv, D), 33, dtype=dtype, count=1)[0]
    q, k = torch.zeros(T, H, D, dtype=dtype, device="cuda"), torch.zeros(T, H_kv, D, dtype=dtype, device="cuda")
    for a, b in zip(cu, cu[1:]):
        for h in range(H):
            q[a:b, h] = ref.huge_inputs(b - a, b - a, D, dtype, 34 + h)[0]
        for h in range(H_kv):
            k[a:b, h] = ref.huge_inputs(b - a, b - a, D, dtype, 36 + h)[1]
    out, lse = attn.attn_fwd_packed(q, k, v, ints(cu), causal=causal, return_lse=True, scale=1.0)
    attn.attn_device_status()
    for a, b in zip(cu, cu[1:]):
        i = torch.arange(b - a, device="cuda")
        visible = i[:, None] >= i if causal else torch.ones(b - a, b - a, dtype=torch.bool, device="cuda")
        for h in range(H):
            g = h * H_kv // H
            ref.check_huge(out[a:b, h], lse[a:b, h], q[a:b, h], k[a:b, g], v[a:b, g], visible, dtype, f"{b - a} head {h}")


def test_a_captured_plan_follows_the_lengths(gpu):
    """40 sequences, planned by a kernel of its own in the call's workspace: two captured
    calls keep theirs apart, and replays take new lengths."""
    T, H, H_kv, D = 4000, 4, 2, 64
    sets = []
    for seed in (40, 41):
        q, k, v = tokens(T, H, H_kv, D, seed, BF16)
        sets.append((q, k, v, ints(offsets([100] * 40)), torch.empty((T, H, D), dtype=BF16, device="cuda")))
    want = [attn.attn_fwd_packed(*x[:4], causal=True) for x in sets]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            attn.attn_fwd_packed(*sets[1][:4], out=sets[1][4], causal=True)
        attn.attn_fwd_packed(*sets[0][:4], out=sets[0][4], causal=True)
        torch.cuda.current_stream().wait_stream(side)
    for lens in (None, [0, 999, 1] * 4 + [0] * 28, [1] * 20 + [199] * 19 + [4000 - 20 - 19 * 199]):
        if lens is not None:
            assert sum(lens) == T and len(lens) == 40
            sets[0][3].copy_(ints(offsets(lens)))
            sets[1][3].copy_(ints(offsets(lens[::-1])))
            want = [attn.attn_fwd_packed(*x[:4], causal=True) for x in sets]
        graph.replay()
        torch.cuda.synchronize()
        attn.attn_device_status()
        assert torch.equal(sets[0][4], want[0]) and torch.equal(sets[1][4], want[1])
