"""What the build makes of a machine: the library needs nvcc alone, the binding's C++
part fits the torch and Python that it was built for (no GPU needed)."""

import os
import subprocess

import pytest

from block_sparse_global_mean_b200 import build as ress_build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build with its products in a folder of its own and its compilers replaced:
    each writes its output, unless it is named in the set that is returned."""
    monkeypatch.setattr(ress_build, "LIB_PATH", str(tmp_path / "libress.so"))
    monkeypatch.setattr(ress_build, "CALL_PATH", str(tmp_path / "_ress_call.so"))
    if hasattr(ress_build, "CALL_TAG_PATH"):
        monkeypatch.setattr(ress_build, "CALL_TAG_PATH", str(tmp_path / "_ress_call.so.tag"))
    broken, made = set(), []

    def run(cmd, check=False, **kw):
        what = "library" if cmd[0] == ress_build._nvcc() else "call"
        made.append(what)
        if what in broken:
            raise subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)

    monkeypatch.setattr(ress_build.subprocess, "run", run)
    return broken, made


def test_the_library_is_built_where_the_binding_cannot_be(elsewhere):
    broken, made = elsewhere
    broken.add("call")
    with pytest.warns(RuntimeWarning, match="ctypes"):
        path = ress_build.build()
    assert path == ress_build.LIB_PATH and os.path.exists(path)
    assert not os.path.exists(ress_build.CALL_PATH)
    broken.clear()
    ress_build.build()
    assert os.path.exists(ress_build.CALL_PATH) and made == ["library", "call", "call"]
    ress_build.build()
    assert made == ["library", "call", "call"]          # nothing is older than its sources


def test_a_library_that_cannot_be_built_is_an_error(elsewhere):
    broken, _ = elsewhere
    broken.add("library")
    with pytest.raises(subprocess.CalledProcessError):
        ress_build.build()


def test_the_binding_is_built_again_for_another_torch(elsewhere, monkeypatch):
    import torch
    broken, made = elsewhere
    ress_build.build()
    monkeypatch.setattr(torch, "__version__", "99.0")
    ress_build.build()
    assert made == ["library", "call", "call"]
    # one that does not fit goes even where it cannot be replaced
    monkeypatch.setattr(torch, "__version__", "99.1")
    broken.add("call")
    with pytest.warns(RuntimeWarning):
        ress_build.build()
    assert not os.path.exists(ress_build.CALL_PATH)


def test_the_binding_refuses_another_torch():
    ress_build.build()
    from block_sparse_global_mean_b200 import ress
    assert ress._call is not None
    with pytest.raises(ImportError, match="built for"):
        ress._call.init(ress.LIB_PATH, "torch 99.0")
