"""A compiled binding that cannot be built or loaded costs time, not the library."""
from __future__ import annotations

import os
import shutil
import sys

import pytest
import torch

import transformer_scaled_dot_fwd_gb300 as attn
from transformer_scaled_dot_fwd_gb300 import build


def test_the_library_is_linked_where_the_binding_does_not_compile(tmp_path, monkeypatch):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    library, out = tmp_path / "lib.so", str(tmp_path / "binding.so")
    for name, value in (("CSRC", str(tmp_path)), ("SOURCES", ["one.cu"]), ("LIB_PATH", str(library)),
                        ("BUILD_DIR", str(tmp_path / "objects"))):
        monkeypatch.setattr(build, name, value)
    fails = [sys.executable, "-c", "print('Python.h: No such file'); raise SystemExit(1)", "-o", out + ".tmp"]
    monkeypatch.setattr(build, "_binding_command", lambda: (out, fails))
    with open(out, "w"):  # a binding of older sources must not stay beside the new library
        os.utime(out, (1, 1))
    with pytest.warns(RuntimeWarning, match="(?s)could not compile csrc/binding.cpp.*Python.h: No such file"):
        assert build.build(quiet=True) == str(library)
    assert library.exists() and not os.path.exists(out)
    # the library is not built again, the binding is tried again
    at = library.stat().st_mtime_ns
    makes = [sys.executable, "-c", f"open({out + '.tmp'!r}, 'w').close()", "-o", out + ".tmp"]
    monkeypatch.setattr(build, "_binding_command", lambda: (out, makes))
    build.build(quiet=True)
    assert library.stat().st_mtime_ns == at and os.path.exists(out)


def test_a_kernel_that_does_not_compile_is_an_error(tmp_path, monkeypatch):
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    (tmp_path / "one.cu").write_text("no code\n")
    for name, value in (("CSRC", str(tmp_path)), ("SOURCES", ["one.cu"]), ("LIB_PATH", str(tmp_path / "lib.so")),
                        ("BUILD_DIR", str(tmp_path / "objects"))):
        monkeypatch.setattr(build, name, value)
    monkeypatch.setattr(build, "_binding_command", lambda: None)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(quiet=True)


@pytest.fixture
def unbound(attn_lib, monkeypatch, tmp_path):
    """The package as it is where no binding was built for the installed torch."""
    monkeypatch.setattr(attn, "_native", None)
    monkeypatch.setattr(attn, "_HERE", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="no compiled binding"):
        attn._load_native()


def test_calls_are_checked_without_the_binding(unbound):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        attn.attn_rope(x, None, torch.zeros(4, dtype=torch.int32), attn.attn_rope_frequencies(64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        attn.attn_fwd_packed(x, x, x, torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["packed", "rope", "rope_append", "tree"])
def test_calls_give_the_same_without_the_binding(gpu, request, name, dtype):
    from test_serving_binding import calls, tensors
    entry, args = calls(dtype=dtype)[name]
    want = [t.clone() for t in tensors(entry(*args))]
    request.getfixturevalue("unbound")
    for kw in ({}, {"stream": torch.cuda.Stream()}):
        torch.cuda.synchronize()
        got = tensors(entry(*args, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_a_depth_of_zero_is_the_library_s_to_refuse(gpu):
    x = torch.zeros(4, 2, 0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(attn.AttnError, match="D must be positive"):
        attn.attn_fwd_packed(x, x.clone(), x.clone(), cu)
    c = torch.zeros(1, 2, 8, 0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(attn.AttnError, match="D must be positive"):
        attn.attn_decode_tree(x.transpose(0, 1)[None], c, c.clone(), cu.new_zeros(4))
