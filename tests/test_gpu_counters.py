"""bf16 prefill launches that run beside each other keep their work counters apart."""
from __future__ import annotations

import ctypes

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def long_call():
    """A call of one work item and some 10 ms, and its result: 128 queries against a
    cache of a million rows."""
    q = wl.random_tensors((1, 1, 128, 64), 80, count=1)[0]
    kc, vc = wl.random_tensors((1, 1, 1 << 20, 64), 81, count=2)
    call = lambda **kw: attn.attn_fwd_chunked(q, kc, vc, **kw)  # noqa: E731
    return call, call()


def short_calls():
    """Calls of one work item, packed and dense, and their results."""
    x = wl.random_tensors((100, 4, 64), 82, count=1)[0]
    cu = ints([0, 60, 100])
    dense = wl.random_tensors((1, 2, 128, 64), 83)
    calls = [lambda **kw: attn.attn_fwd_packed(x[:, :2], x[:, 2:3], x[:, 3:], cu, causal=True, **kw),
             lambda **kw: attn.attn_fwd(*dense, causal=True, **kw)]
    return [(c, c()) for c in calls]


def test_a_long_call_beside_many_short_ones(gpu):
    """300 short calls on each of two streams while a long one runs on a third."""
    (call, want), shorts = long_call(), short_calls()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    with torch.cuda.stream(s[0]):
        long_out = call(stream=s[0])
    got = []
    for i in range(600):
        c, w = shorts[i // 2 % 2]
        with torch.cuda.stream(s[1 + i % 2]):
            got.append((c(stream=s[1 + i % 2]), w))
    torch.cuda.synchronize()
    attn.attn_device_status()
    assert torch.equal(long_out, want)
    for a, b in got:
        assert torch.equal(a, b)


def test_many_short_calls_behind_a_long_one(gpu):
    """In one stream: each is placed as soon as the one before it has started, so many
    wait beside the long call for its end."""
    (call, want), shorts = long_call(), short_calls()
    torch.cuda.synchronize()
    got = [(call(), want)]
    for i in range(300):
        c, w = shorts[i % 2]
        got.append((c(), w))
    got.append((call(), want))
    torch.cuda.synchronize()
    attn.attn_device_status()
    for a, b in got:
        assert torch.equal(a, b)


def test_more_streams_than_counters(gpu):
    """Streams come and go: a new one takes the counter of one that is long done."""
    shorts = short_calls()
    cudart = torch.cuda.cudart()
    handles = []
    for i in range(600):
        c, w = shorts[i % 2]
        if i % 2:
            handles.append(ctypes.c_void_p())
            assert int(cudart.cudaStreamCreate(ctypes.addressof(handles[-1]))) == 0
            s = torch.cuda.ExternalStream(handles[-1].value)
        else:
            s = torch.cuda.ExternalStream(handles[i // 4].value) if handles else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(w)
        c(out=out, stream=s)
        s.synchronize()
        assert torch.equal(out, w)
    attn.attn_device_status()
    for h in handles:
        assert int(cudart.cudaStreamDestroy(h.value)) == 0
