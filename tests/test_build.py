"""The build of the binding's marshalling: left out where torch was built without CUDA, and made again
for another torch (no GPU)."""
import os
import types

import pytest

from activation_epilogue_gb300 import build as libbuild


@pytest.fixture
def torch_tree(tmp_path, monkeypatch):
    """A torch folder with the headers that both kinds of torch have, in place of the real one; the
    products go to tmp_path."""
    root = tmp_path / "torch"
    header = root / "include" / "torch" / "csrc" / "autograd" / "python_variable.h"
    header.parent.mkdir(parents=True)
    header.write_text("")
    (root / "lib").mkdir()
    for name in ("torch_python", "torch_cpu", "c10"):
        (root / "lib" / f"lib{name}.so").write_text("")
    (root / "version.py").write_text("__version__ = '1+cpu'\n")
    find = libbuild.importlib.util.find_spec
    monkeypatch.setattr(libbuild.importlib.util, "find_spec", lambda name: types.SimpleNamespace(
        submodule_search_locations=[str(root)]) if name == "torch" else find(name))
    for name in ("FASTCALL", "FASTCALL_STAMP"):
        monkeypatch.setattr(libbuild, name, str(tmp_path / name.lower()), raising=False)
    return root


def _with_cuda(root):
    header = root / "include" / "c10" / "cuda" / "CUDAStream.h"
    header.parent.mkdir(parents=True)
    header.write_text("")
    (root / "lib" / "libc10_cuda.so").write_text("")


def test_a_torch_without_cuda_leaves_the_marshalling_out(torch_tree):
    libbuild._compile_fastcall()         # (g++ would fail on this tree: it is not asked)
    assert libbuild._fastcall_paths() is None
    assert not os.path.exists(libbuild.FASTCALL)
    assert not libbuild._fastcall_stale()


def test_the_marshalling_of_a_torch_that_is_gone_goes_too(torch_tree):
    with open(libbuild.FASTCALL, "w") as fh:
        fh.write("built for another torch")
    assert libbuild._fastcall_stale()
    libbuild._compile_fastcall()
    assert not os.path.exists(libbuild.FASTCALL)


def test_another_torch_makes_the_marshalling_stale(torch_tree, monkeypatch):
    _with_cuda(torch_tree)
    assert libbuild._fastcall_paths() is not None and libbuild._fastcall_stale()

    def compiler(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as fh:
            fh.write("product")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(libbuild.subprocess, "run", compiler)
    libbuild._compile_fastcall()
    assert not libbuild._fastcall_stale()
    (torch_tree / "version.py").write_text("__version__ = '2+cu'\n")
    assert libbuild._fastcall_stale()
    libbuild._compile_fastcall()
    assert not libbuild._fastcall_stale()
