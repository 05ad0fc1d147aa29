"""What build() takes for current: the library by its sources, and the quick way in by its sources and the installed
torch, whose modules never outlive the library they were built beside."""

import os

import pytest
import torch

from mxfp8_block_scaled_inv_gb300 import build


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A build whose commands write their outputs and do nothing else."""
    here, csrc = tmp_path / "pkg", tmp_path / "csrc"
    here.mkdir()
    csrc.mkdir()
    for f in (*build.CU_SOURCES, *build.CXX_SOURCES, "fastcall.cpp"):
        (csrc / f).write_text("")
    ran, broken = [], set()

    def run(cmd, verbose):
        out = os.path.basename(cmd[cmd.index("-o") + 1])
        ran.append(out)
        if any(b in out for b in broken):
            raise RuntimeError(f"cannot make {out}")
        with open(cmd[cmd.index("-o") + 1], "wb"):
            pass
        return ""

    monkeypatch.setattr(build, "HERE", str(here))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(here / "libmxq.so"))
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_tried", set(), raising=False)
    # Everything that is there is old, as it is for a checkout that was built.
    for f in (*csrc.iterdir(),):
        os.utime(f, (1, 1))
    return type("Tree", (), dict(here=here, csrc=csrc, ran=ran, broken=broken,
                                 fast=staticmethod(lambda v=torch.__version__: build.fastcall_path(v))))


def touch(path, when=None):
    open(path, "wb").close()
    if when is not None:
        os.utime(path, (when, when))


def test_everything_is_built_once(tree):
    build.build()
    assert os.path.exists(build.LIB_PATH) and os.path.exists(tree.fast())
    assert len(tree.ran) == len(build.CU_SOURCES) + len(build.CXX_SOURCES) + 2
    tree.ran.clear()
    build.build()
    assert tree.ran == []
    build.build(force=True)
    assert len(tree.ran) == len(build.CU_SOURCES) + len(build.CXX_SOURCES) + 2 and os.path.exists(tree.fast())


def test_another_torch_gets_its_module_beside_a_current_library(tree):
    touch(build.LIB_PATH)
    touch(tree.fast("0.1"))  # that of the torch before
    build.build()
    assert tree.ran == [os.path.basename(tree.fast()) + ".tmp"]
    assert os.path.exists(tree.fast()) and os.path.exists(tree.fast("0.1"))
    touch(tree.fast(), when=1)  # older than the sources
    tree.ran.clear()
    build.build()
    assert tree.ran == [os.path.basename(tree.fast()) + ".tmp"]


def test_a_new_library_takes_the_modules_of_the_old_one_away(tree, monkeypatch):
    touch(build.LIB_PATH, when=1)
    for v in ("0.1", torch.__version__):
        touch(tree.fast(v))
    import sys

    monkeypatch.setitem(sys.modules, "torch", None)  # not to be imported: no module of its own
    build.build()
    assert [f for f in os.listdir(tree.here) if f.startswith("mxq_fastcall")] == []
    assert os.path.exists(build.LIB_PATH)


def test_a_module_that_cannot_be_built(tree, capsys):
    touch(build.LIB_PATH)
    touch(tree.fast(), when=1)
    tree.broken.add("mxq_fastcall")
    for _ in range(2):
        assert build.build() == build.LIB_PATH
    assert len(tree.ran) == 1 and not os.path.exists(tree.fast())  # tried once, and the older one is gone
    assert "mxq_fastcall not built" in capsys.readouterr().err
    tree.broken.clear()
    build.build(force=True)
    assert os.path.exists(tree.fast())


def test_no_module_without_its_library(tree):
    touch(build.LIB_PATH, when=1)
    tree.broken.add("libmxq")
    with pytest.raises(RuntimeError):
        build.build()
    assert not os.path.exists(tree.fast())
