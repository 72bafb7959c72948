"""The compiled binding of the serving calls (csrc/binding.cpp): it answers the
usual call as the checked path in Python does, and leaves every other call to
that path by answering None, before it writes anything."""
import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn


@pytest.fixture(scope="module")
def native(attn_lib):
    return attn._native or attn._load_native()


def calls(device="cuda", dtype=torch.bfloat16):
    """name -> (entry point, native function, its arguments in order)."""
    g = torch.Generator().manual_seed(5)
    T, H, H_kv, D, B, Skv = 37, 4, 2, 64, 2, 96

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dtype).to(device)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device=device)

    x = rnd(T, H + 2 * H_kv, D)
    q, k, v = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    kc, vc = rnd(B, H_kv, Skv, D), rnd(B, H_kv, Skv, D)
    fr = attn.attn_rope_frequencies(D)
    return {
        "packed": (attn.attn_fwd_packed, [q, k, v, ints(0, 30, 37), None, None, None, True, True]),
        "rope": (attn.attn_rope, [q, k, ints(*range(T)), fr, None, None, False, False, 1.0]),
        "rope_append": (attn.attn_rope_append,
                        [q, k, v, kc, vc, fr, ints(0, 30, 37), ints(60, 90), None, None, torch.empty_like(k), True, 1]),
        "tree": (attn.attn_decode_tree,
                 [rnd(B, 8, H, D).transpose(1, 2), kc, vc, ints(-1, 0, 0, 1, 1, 2, 2, 5), ints(50, 96), None, None, None]),
    }


def tensors(r):
    return list(r) if isinstance(r, tuple) else [r]


@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_none_for_what_is_not_on_the_device(native, name):
    f = getattr(native, name)
    args = calls(device="cpu")[name][1]
    assert f(*args) is None
    assert f(*[None] * len(args)) is None and f(*["x"] * len(args)) is None
    assert f() is None and f(*args, None) is None
    with pytest.raises(ValueError, match="CUDA tensor"):
        calls(device="cpu")[name][0](*args)


def test_bind_refuses_bad_addresses(native):
    for bad in ((), (1,) * 5, (0,) * 6):
        with pytest.raises((TypeError, ValueError)):
            native.bind(*bad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_same_as_the_checked_path(native, name, dtype):
    entry, args = calls(dtype=dtype)[name]
    caches = args[3:5] if name == "rope_append" else []
    got = getattr(native, name)(*args)
    assert got is not None
    got = [t.clone() for t in tensors(got) + caches]
    want = [t.clone() for t in tensors(entry(*args, stream=torch.cuda.current_stream())) + caches]
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.shape == b.shape and a.stride() == b.stride() and a.dtype == b.dtype
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_given_outputs_are_returned(native, name):
    _, args = calls()[name]
    first = tensors(getattr(native, name)(*args))
    out = [torch.full_like(t, 7) for t in first]
    at = {"packed": (4, 5), "rope": (4, 5), "rope_append": (9, 10), "tree": (6,)}[name]
    for i, t in zip(at, out):
        args[i] = t
    again = tensors(getattr(native, name)(*args))
    for a, b, t in zip(first, again, out):
        assert b is t and torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_other_calls_are_left_to_the_checked_path(native, name):
    entry, args = calls()[name]
    f = getattr(native, name)

    class Sub(torch.Tensor):
        pass

    last = {"packed": 7, "rope": 6, "rope_append": 11, "tree": 7}[name]
    changes = [(0, args[0].float()), (0, args[0].half()), (0, args[0][..., :32]), (0, args[0][0]), (0, args[0].cpu()),
               (0, args[0].as_subclass(Sub)), (1, args[1].float()), (1, args[1][..., ::2]), (1, args[1][:1]),
               (last, "x"), (last, 1j)]
    changes += {
        "packed": lambda: [(2, args[2][:, :1]), (3, args[3].long()), (3, args[3][:0]), (4, args[0][:5]), (5, args[0]),
                           (5, torch.empty(37, 4, device="cuda").double()), (7, 1)],
        "rope": lambda: [(2, None), (2, args[2][:5]), (3, args[3].float()), (3, args[3].repeat(9)), (3, args[3].cuda()),
                         (4, args[0][:5]), (5, args[0]), (8, None), (7, 0)],
        "rope_append": lambda: [(2, args[2][:, :1]), (3, args[3][:1]), (4, args[4].transpose(1, 2)), (5, None),
                                (6, args[6][:2]), (7, args[7].long()), (8, args[7]), (10, args[0]), (12, None)],
        "tree": lambda: [(1, args[1][:1]), (2, args[2].transpose(1, 2)), (3, args[3][:3]), (4, args[4][:1]),
                         (5, args[4].long()), (6, args[0][:1]), (7, float("nan"))],
    }[name]()
    for i, bad in changes:
        assert f(*args[:i], bad, *args[i + 1:]) is None, (i, bad)
    assert f(*args) is not None
    # refusals of the library, by the checked path's exception
    with pytest.raises(attn.AttnError):
        if name in ("rope", "rope_append"):
            entry(*args[:-1], float("inf"))
        elif name == "packed":
            entry(*args[:6], float("inf"), True, True)
        else:
            entry(*args[:7], float("inf"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_the_checked_path_gives_the_same(native, name, dtype):
    # integers for flags, a float of another type: valid, but not the usual call
    class Float(float):
        pass

    entry, args = calls(dtype=dtype)[name]
    i, other = {"packed": (7, 1), "rope": (6, 0), "rope_append": (11, 1), "tree": (7, Float(64 ** -0.5))}[name]
    unusual = args[:i] + [other] + args[i + 1:]
    assert getattr(native, name)(*unusual) is None
    caches = args[3:5] if name == "rope_append" else []
    got = [t.clone() for t in tensors(entry(*args)) + caches]
    for t in caches:
        t.zero_()
    want = tensors(entry(*unusual)) + caches
    if caches:  # rows that are not written were zeroed
        for a, b in zip(got[-2:], caches):
            a[b == 0] = 0
    for a, b in zip(got, want):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.gpu
def test_parameters_and_other_threads(native):
    import threading
    entry, args = calls()["rope"]
    want = tensors(entry(*args))
    args[1] = torch.nn.Parameter(args[1].clone(), requires_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(tensors(entry(*args)), want))
    got = [[] for _ in range(4)]

    def work(out):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                out[:] = tensors(entry(*args))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(g,)) for g in got]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_captured(native, name, dtype):
    """The same call captured twice into one graph, after an eager one on another
    stream, and replayed: the eager results (fp32: clusters of CTAs in a graph)."""
    entry, args = calls(dtype=dtype)[name]
    want = [t.clone() for t in tensors(entry(*args))]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        entry(*args)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = tensors(entry(*args))
        second = tensors(entry(*args))
    for _ in range(3):
        for t in first + second:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, first, second):
            assert torch.equal(a, b) and torch.equal(a, c)
    attn.attn_device_status()
