"""The build without a torch that the native binding can be made against, and after an
update of torch."""
import os
import sys
import types

import pytest

from block_sparse_long_10_b200 import build as qbuild


@pytest.fixture
def bind(tmp_path, monkeypatch):
    """The binding's place in an empty folder, and what is linked to it."""
    qbuild.build()  # the library itself is up to date
    linked = []

    def link(cmd, out, verbose):
        assert cmd
        linked.append(out)
        open(out, "w").close()

    monkeypatch.setattr(qbuild, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(qbuild, "BIND_STAMP", str(tmp_path / "stamp"), raising=False)
    monkeypatch.setattr(qbuild, "_link", link)
    return linked


def test_the_library_builds_without_torch(bind, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert qbuild.build() == qbuild.LIB
    assert bind == [] and not os.path.exists(qbuild.BIND)


def test_the_library_builds_with_a_torch_without_cuda(bind, monkeypatch, tmp_path):
    torch = types.SimpleNamespace(__file__=str(tmp_path / "torch" / "__init__.py"),
                                  __version__="1.0+cpu",
                                  _C=types.SimpleNamespace(_GLIBCXX_USE_CXX11_ABI=True))
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert qbuild.build() == qbuild.LIB
    assert bind == [] and not os.path.exists(qbuild.BIND)


def test_the_binding_is_built_once_for_a_torch_and_again_for_another(bind, monkeypatch):
    import torch
    qbuild.build()
    qbuild.build()
    assert bind == [qbuild.BIND]
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    qbuild.build()
    qbuild.build()
    assert bind == [qbuild.BIND] * 2
    monkeypatch.setitem(sys.modules, "torch", None)
    qbuild.build()  # one for a torch that has gone is not left behind
    assert bind == [qbuild.BIND] * 2 and not os.path.exists(qbuild.BIND)
