"""When the native module is built again, and what the library needs it for: with
stand-ins for the compilers."""
import os
import sys
import types

import pytest
import torch

import top_routed_grouped_gb300 as moe
from top_routed_grouped_gb300 import build, train


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs in a folder of their own; compilers that write what -o names, or fail."""
    for name, file in (("BUILD", "_build"), ("LIB", "lib.so"), ("BIND", "_tensor_list.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    log = tmp_path / "calls"

    def compiler(name, ok=True):
        path = tmp_path / name
        path.write_text("#!/bin/sh\n" f"echo {name} >> {log}\n" + (
            'while [ $# -gt 0 ]; do [ "$1" = -o ] && touch "$2"; shift; done\n' if ok else "exit 1\n"))
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(build, "_nvcc", lambda: compiler("nvcc"))
    monkeypatch.setenv("CXX", compiler("cxx"))
    calls = lambda: log.read_text().split().count("cxx") if log.exists() else 0  # noqa: E731
    return types.SimpleNamespace(calls=calls, broken=lambda: monkeypatch.setenv("CXX", compiler("broken", ok=False)))


def test_the_module_is_built_again_for_another_torch_or_python(tree, monkeypatch):
    build.build()
    assert tree.calls() == 1
    build.build()
    build.build_bind()
    assert tree.calls() == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert tree.calls() == 2
    build.build()
    assert tree.calls() == 2
    os.remove(build.BIND)
    build.build()
    assert tree.calls() == 3


def test_the_library_is_there_without_the_module(tree, monkeypatch):
    tree.broken()
    with pytest.raises(RuntimeError, match="broken"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    os.remove(build.LIB)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.BIND)


@pytest.mark.parametrize("module", [None, types.SimpleNamespace(pack=None), types.SimpleNamespace(pack=None, built_for="")])
def test_a_module_of_another_torch_is_not_used(monkeypatch, module):
    name = "top_routed_grouped_gb300._tensor_list"
    monkeypatch.delattr(moe, "_tensor_list", raising=False)
    monkeypatch.setitem(sys.modules, name, module)
    if module is not None:
        monkeypatch.setattr(moe, "_tensor_list", module, raising=False)
    with pytest.raises(RuntimeError, match="top_routed_grouped_gb300.build"):
        train._packer()


def test_the_module_that_is_there_is_of_this_torch():
    from top_routed_grouped_gb300 import _tensor_list
    assert _tensor_list.built_for == build.bind_target() and train._packer() is _tensor_list.pack
