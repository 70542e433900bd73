"""Building and loading the native front of the serving operators, without a GPU."""

import os

import pytest

import post_weight_quantization_layer_b200.build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build directory of its own, with a library and a front newer than their sources."""
    for name, file in (("LIBDIR", ""), ("LIB", "libgptq.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(B, name, str(tmp_path / file))
    (tmp_path / "libgptq.so").write_text("library")
    (tmp_path / "_binding.so").write_text("front")
    return tmp_path


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
