"""The build without a compiler: what is built when torch is there, when it is
not, and when it has changed (CPU; compilers are stood in for)."""
import os
import subprocess
import sys
import types

import pytest

from sparse_reuse_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of its own whose compilers write the file after -o."""
    ran = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("x")
        ran.append(os.path.basename(out))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in (*build.SOURCES, "sf_torch.cpp"):
        (csrc / name).write_text("")
        os.utime(csrc / name, (1, 1))
    for name, value in (("CSRC", csrc), ("INCLUDE", csrc), ("BUILD", tmp_path / "_build"), ("PKG", tmp_path),
                        ("LIB", tmp_path / "libspecfold.so"), ("TORCH_EXT", tmp_path / "_sf_torch.so"),
                        ("TORCH_STAMP", tmp_path / "_build" / "sf_torch.version")):
        monkeypatch.setattr(build, name, str(value), raising=False)
    monkeypatch.setattr(build, "_inputs", lambda: [str(csrc / n) for n in (*build.SOURCES, "sf_torch.cpp")])
    monkeypatch.setattr(subprocess, "run", run)
    return types.SimpleNamespace(path=tmp_path, ran=ran)


def test_without_torch_the_library_alone_is_built(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_EXT)
    assert build.up_to_date()
    n = len(tree.ran)
    build.build()
    assert len(tree.ran) == n                            # nothing left to do
    monkeypatch.undo()


def test_a_torch_that_appears_or_changes_is_built_for(tree, monkeypatch):
    import torch
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        build.build()
    assert not build.up_to_date()
    build.build()
    assert os.path.exists(build.TORCH_EXT) and build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert not build.up_to_date()
        tree.ran.clear()
        build.build()
        assert "_sf_torch.so.tmp" in tree.ran and build.up_to_date()
    assert not build.up_to_date()


def test_without_python_headers_the_library_alone_is_built(tree, monkeypatch):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tree.path / "none")})
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_EXT) and build.up_to_date()


def test_a_changed_source_is_built(tree):
    build.build()
    assert build.up_to_date()
    src = os.path.join(build.CSRC, build.SOURCES[0])
    os.utime(src, (1 << 33, 1 << 33))
    assert not build.up_to_date()
