"""Building and loading the native front of the serving operators, without a GPU."""

import os

import pytest

import post_weight_quantization_layer_b200.build as B
from post_weight_quantization_layer_b200 import _native


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build directory of its own, with a library and a front newer than their sources."""
    for name, file in (("LIBDIR", ""), ("LIB", "libgptq.so"), ("BINDING", "_binding.so"), ("BINDING_ABI", "_binding.abi")):
        monkeypatch.setattr(B, name, str(tmp_path / file))
    (tmp_path / "libgptq.so").write_text("library")
    (tmp_path / "_binding.so").write_text("front")
    (tmp_path / "_binding.abi").write_text(B.binding_abi() + "\n")
    return tmp_path


def test_a_front_for_another_torch_is_built_again_and_not_loaded(tree, monkeypatch):
    assert not B.needs_build() and not B.binding_needs_build()
    monkeypatch.setattr(_native, "_binding", None)
    monkeypatch.setattr(_native, "BINDING_PATH", B.BINDING)
    for record in ("torch 2.0.0 cxx11 0 cpython-38-x86_64-linux-gnu\n", None):
        if record is None:
            os.unlink(B.BINDING_ABI)
        else:
            (tree / "_binding.abi").write_text(record)
        assert B.binding_needs_build() and not B.needs_build()
        with pytest.raises(RuntimeError, match="was built for"):
            _native.binding()


def test_the_record_follows_a_build(tree, monkeypatch):
    os.unlink(B.BINDING_ABI)
    monkeypatch.setattr(B, "binding_command", lambda out: ["sh", "-c", f"echo new > {out}"])
    assert B.build() == B.LIB
    assert (tree / "_binding.so").read_text() == "new\n" and (tree / "libgptq.so").read_text() == "library"
    assert not B.binding_needs_build()


@pytest.mark.parametrize("front", [["sh", "-c", "echo no headers >&2; exit 3"], ["no-such-compiler"]])
def test_the_library_is_installed_where_the_front_cannot_be_built(tree, monkeypatch, front):
    os.unlink(B.LIB)
    os.unlink(B.BINDING)
    (tree / "nvcc").write_text('#!/bin/sh\nfor a; do out=$a; done\necho built > "$out"\n')
    (tree / "nvcc").chmod(0o755)
    monkeypatch.setattr(B, "nvcc", lambda: str(tree / "nvcc"))
    monkeypatch.setattr(B, "binding_command", lambda out: front)
    with pytest.raises(RuntimeError, match="_binding.so"):
        B.build()
    assert (tree / "libgptq.so").read_text() == "built\n" and not os.path.exists(B.BINDING)


def test_without_the_front_the_wrappers_check_and_call_themselves(tree, monkeypatch):
    import torch

    import post_weight_quantization_layer_b200 as gq

    for path in (str(tree / "nothing.so"), B.BINDING):  # not there; not a library
        monkeypatch.setattr(_native, "_binding", None)
        monkeypatch.setattr(_native, "_front", None)
        monkeypatch.setattr(_native, "BINDING_PATH", path)
        kv, slots = torch.zeros(3, 2, 64).bfloat16(), torch.zeros(3, dtype=torch.int32)
        cache = gq.new_cache(1, 2, 64, 16, 8, device="cpu")
        with pytest.warns(RuntimeWarning, match="go through ctypes"):
            with pytest.raises(ValueError, match="CUDA tensors"):
                gq.cache_write(kv, kv, cache, slots, 8)
        with pytest.raises(ValueError, match="bits must be"):
            gq.cache_read(cache, slots, 5)


def test_a_step_without_tokens():
    import torch

    from post_weight_quantization_layer_b200 import serving

    batch = serving.step_batch([[3], []], [5, 0], [0, 0], 16, device="cpu")
    layer = serving.ServedLayer({}, (), 4, 2, torch.zeros(32, dtype=torch.float64))
    out = serving.decoder_layer_step(torch.zeros(0, 256).bfloat16(), layer, {}, batch)
    assert out.shape == (0, 256) and out.dtype == torch.bfloat16
    with pytest.raises(ValueError, match="width"):
        serving.step_batch([[], []], [0, 0], [0, 0], 16, device="cpu", width=0)
