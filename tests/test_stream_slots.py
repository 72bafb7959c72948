"""The work counters of bf16 prefill calls (csrc/stream_slots.h, compiled here for the
CPU): two launches may only share a counter when their stream orders them."""
from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N = 8
SOURCE = """
#include "stream_slots.h"
static attn::StreamSlots<%d> slots;
extern "C" int slot_of(unsigned long long stream) { return slots.of(stream); }
extern "C" void forget() { slots = attn::StreamSlots<%d>(); }
""" % (N, N)


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("slots")
    (d / "s.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "transformer_scaled_dot_fwd_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-shared", "-fPIC", "-I", csrc, str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    handle = ctypes.CDLL(str(d / "s.so"))
    handle.slot_of.argtypes = [ctypes.c_ulonglong]
    return handle


def test_a_long_call_keeps_its_counter(slots):
    """However many calls other streams make while one of its calls runs."""
    slots.forget()
    first = slots.slot_of(1)
    assert all(slots.slot_of(2 + i % 3) != first for i in range(10000))
    assert slots.slot_of(1) == first


def test_streams_in_use_never_share(slots):
    """Any order of calls by as many streams as there are slots."""
    slots.forget()
    r = random.Random(1)
    ids = r.sample(range(1 << 60), N)
    slot = {}
    for _ in range(5000):
        i = r.choice(ids)
        assert slot.setdefault(i, slots.slot_of(i)) == slots.slot_of(i)
    assert sorted(slot.values()) == sorted(set(slot.values())) and set(slot.values()) <= set(range(N))


def test_the_idle_stream_gives_way(slots):
    """One stream more than slots takes the slot of the one unused for the longest time."""
    slots.forget()
    r = random.Random(2)
    order, slot = [], {}
    for _ in range(5000):
        i = r.choice(order[-4:]) if order and r.random() < 0.5 else r.randrange(3 * N)
        s = slots.slot_of(i)
        if i in slot:
            assert s == slot[i]
            order.remove(i)
        elif len(order) == N:
            assert s == slot.pop(order.pop(0))
        else:
            assert s not in slot.values()
        order.append(i)
        slot[i] = s


def test_tags_tell_near_launches_apart():
    """The sum of up to 152 tags of one launch is no multiple of another's tag within
    13000 launches, so the first draw that meets them shows the conflict."""
    base = 1 << 21
    r = random.Random(3)
    for _ in range(400):
        turn, apart = r.randrange(base), r.choice((1, 2, 13000, r.randint(1, 13000)))
        a, b = base + turn, base + (turn + apart) % base
        if abs(a - b) > 13000:
            continue  # the turn began again: any two tags
        assert all(n * a % b and n * b % a for n in range(1, 153))
    assert 1024 * (2 * base - 1) < 1 << 32
