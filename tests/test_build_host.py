"""The build on the CPU, with a stand-in for nvcc: the C library does not depend on what the Python
binding needs, and a binding made for another torch or Python is made again."""
import os
import sys

import pytest

import sparse_moe_layer_gb300 as moe

B = sys.modules["sparse_moe_layer_gb300.build"]  # (the package's `build` is the function)

NVCC = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo built > "$2"; fi
  shift
done
for mx in 0 1; do
  echo "Compiling entry function '_ZN3moe15moe_gemm_kernelILb${mx}Ex' for sm_103a"
  echo "Used 168 registers"
done >&2
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    bin_ = tmp_path / "cuda" / "bin"
    bin_.mkdir(parents=True)
    (bin_ / "nvcc").write_text(NVCC)
    (bin_ / "nvcc").chmod(0o755)
    monkeypatch.setenv("CUDA_HOME", str(tmp_path / "cuda"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "binding.so"))
    made = []

    def compile_binding():
        made.append(1)
        return "binding.o"

    def link_binding(obj):
        assert os.path.exists(B.LIB)  # it links against the library
        open(B.BINDING, "w").close()
        with open(B._stamp(), "w") as f:
            f.write(B._binding_made_for())

    monkeypatch.setattr(B, "_compile_binding", compile_binding)
    monkeypatch.setattr(B, "_link_binding", link_binding)
    return made


def test_both_are_built_once(tree):
    assert B.build() == B.LIB and os.path.exists(B.BINDING) and tree == [1]
    before = os.path.getmtime(B.LIB)
    B.build()
    assert tree == [1] and os.path.getmtime(B.LIB) == before


@pytest.mark.parametrize("what", ["g++", "Python.h", "torch's headers"])
def test_the_library_needs_nvcc_only(tree, monkeypatch, what):
    monkeypatch.setattr(B, "_binding_missing", lambda: what)
    with pytest.warns(UserWarning, match="no Python entries"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not tree and not os.path.exists(B.BINDING)


def test_a_binding_that_fails_leaves_the_library(tree, monkeypatch):
    def broken():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(B, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_a_binding_for_another_torch_is_made_again(tree, monkeypatch):
    B.build()
    before = os.path.getmtime(B.LIB)
    monkeypatch.setattr(B, "_binding_made_for", lambda: "torch 0.0 python 3")
    assert not B.binding_current()
    with monkeypatch.context() as m:
        m.setattr(moe, "_calls", None)
        m.setattr(moe, "lib", lambda: None)
        with pytest.raises(RuntimeError, match="not built for this torch"):
            moe._entries()
    B.build()
    assert tree == [1, 1] and B.binding_current() and os.path.getmtime(B.LIB) == before
