"""The compiled binding of the calls of a paged cache answers the usual call as the checked
path in Python does, returns the outputs it is given, and leaves every other call to that
path before it writes anything."""
from __future__ import annotations

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn

pytestmark = pytest.mark.gpu
NAMES = ["paged", "paged ragged", "norm_rope", "append_paged", "pages_step", "pages_compact"]


@pytest.fixture(scope="module")
def native(attn_lib):
    f = attn._native or attn._load_native()
    if isinstance(f, attn._NoBinding):
        pytest.skip("no binding")
    return f


def calls(dtype=torch.bfloat16):
    """name -> (entry point, native function's name, its arguments in order, tensors written)."""
    g = torch.Generator().manual_seed(5)
    H, H_kv, D, P, n_pages = 4, 2, 64, 16, 40

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dtype).cuda()

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    kp, vp = rnd(n_pages, H_kv, P, D), rnd(n_pages, H_kv, P, D)
    table, lens, cu = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()[:30].view(3, 10), ints(60, 7, 150), ints(0, 30, 31, 37)
    x = rnd(37, H + 2 * H_kv, D)
    q, k, v = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    f, w = attn.attn_rope_frequencies(D), rnd(D)
    return {
        "paged": (attn.attn_fwd_paged, "paged", [rnd(3, H, D), kp, vp, table, lens, None, None, None, None, False], []),
        "paged ragged": (attn.attn_fwd_paged, "paged", [q, kp, vp, table, lens, cu, None, None, 0.3, True], []),
        "norm_rope": (attn.attn_norm_rope, "norm_rope", [q, k, ints(*range(37)), f, w, None, 1e-5, None, None, True, 1.0], []),
        "append_paged": (attn.attn_rope_append_paged, "append_paged",
                         [q, k, v, kp, vp, table, f, lens, cu, None, None, w, 1e-5, None, torch.empty_like(k), False, 1], [kp, vp]),
        "pages_step": (attn.attn_pages_step, "pages_step", [table, lens, n_pages, P, ints(0, 0, 2, -1), ints(61, 61, 3, 20), None, None], []),
        "pages_compact": (attn.attn_pages_compact, "pages_compact", [table, lens, n_pages, P, ints(*([0] * 39 + [1])), None], []),
    }


def tensors(r):
    return list(r) if isinstance(r, tuple) else [r]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", NAMES)
def test_same_as_the_checked_path(native, name, dtype):
    entry, fast, args, written = calls(dtype)[name]
    got = getattr(native, fast)(*args)
    assert got is not None
    got = [t.clone() for t in tensors(got) + written]
    want = [t.clone() for t in tensors(entry(*args, stream=torch.cuda.current_stream())) + written]
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.shape == b.shape and a.stride() == b.stride() and a.dtype == b.dtype and torch.equal(a, b)


def test_given_outputs_are_returned(native):
    _, _, args, _ = calls()["paged ragged"]
    out, lse = torch.empty_like(args[0].contiguous()), torch.empty(37, 4, device="cuda")
    args[6], args[7] = out, lse
    got = native.paged(*args)
    assert got[0] is out and got[1] is lse
    _, _, args, _ = calls()["norm_rope"]
    args[7] = torch.empty(37, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert native.norm_rope(*args)[0] is args[7]


def test_pages_are_copied(native):
    _, _, args, _ = calls()["append_paged"]
    kp, vp = args[3], args[4]
    c = torch.tensor([[3, 5, 16], [1, 2, 4]], dtype=torch.int32, device="cuda")
    want = [x.clone() for x in (kp, vp)]
    for x in want:
        x[5] = x[3]
        x[2, :, :4] = x[1, :, :4]
    assert native.pages_copy(kp, vp, c) is True
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert native.pages_copy(kp[None], vp[None], c) is True and native.pages_copy(kp, vp[:3], c) is None


@pytest.mark.parametrize("name,position,value", [
    ("paged", 4, torch.ones(3)), ("paged", 5, torch.ones(2, dtype=torch.int32)), ("paged", 3, torch.zeros(3, 10)),
    ("norm_rope", 4, torch.ones(3)), ("append_paged", 11, torch.ones(64, dtype=torch.float64)), ("pages_step", 2, 3.0),
    ("pages_step", 7, ()), ("pages_compact", 4, torch.ones(40))])
def test_other_calls_are_left(native, name, position, value):
    _, fast, args, written = calls()[name]
    args[position] = value.cuda() if torch.is_tensor(value) else value
    before = [t.clone() for t in written]
    assert getattr(native, fast)(*args) is None
    assert all(torch.equal(a, b) for a, b in zip(before, written))


def test_refusals_of_the_checked_path(native):
    """What the binding leaves, with its reason."""
    c = calls()
    for name, position, value, error in (("paged", 0, "half", TypeError), ("paged", 3, "table", ValueError), ("append_paged", 11, "w", TypeError),
                                         ("paged ragged", 5, "cu", ValueError)):
        entry, _, args, _ = c[name]
        args = list(args)
        args[position] = {"half": args[0].half(), "table": torch.zeros(3, 10, device="cuda"), "w": torch.ones(64, device="cuda"),
                          "cu": torch.zeros(9, dtype=torch.int32, device="cuda")}[value]
        with pytest.raises(error):
            entry(*args)
    with pytest.raises(attn.AttnError) as e:  # a page size of 12 rows
        attn.attn_fwd_paged(c["paged"][2][0], *(torch.zeros(4, 2, 12, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)),
                            torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    assert e.value.code == attn.ATTN_EUNSUPPORTED
