"""The build: what one part's failure leaves of the others, and what is made again."""
import os

import pytest

from fp4_block_scaled_quantize_gb300 import build as fbuild


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small unit into a folder of its own."""
    for name in ("BUILD", "LIBDIR"):
        monkeypatch.setattr(fbuild, name, str(tmp_path / name))
    monkeypatch.setattr(fbuild, "LIB", str(tmp_path / "LIBDIR" / "libfp4gb300.so"))
    monkeypatch.setattr(fbuild, "BIND", str(tmp_path / "LIBDIR" / "_bind.so"))
    monkeypatch.setattr(fbuild, "UNITS", {"abi.cu": []})


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler"])
def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch, cxx):
    """A host compiler or torch headers that fail are reported, after the CUDA
    library, which needs neither, is there; no older binding stays beside it."""
    os.makedirs(fbuild.LIBDIR)
    open(fbuild.BIND, "w").close()
    monkeypatch.setenv("CXX", cxx)
    with pytest.raises(RuntimeError, match="bind.cpp"):
        fbuild.build()
    assert os.path.exists(fbuild.LIB) and not os.path.exists(fbuild.BIND)


def test_the_binding_is_made_again_for_another_torch(elsewhere, monkeypatch):
    """It is compiled against torch's C++ headers: another torch, or another
    interpreter, means another binding."""
    import torch
    fbuild.build()
    first = os.stat(fbuild.BIND).st_mtime_ns
    fbuild.build()
    assert os.stat(fbuild.BIND).st_mtime_ns == first
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".another")
    fbuild.build()
    second = os.stat(fbuild.BIND).st_mtime_ns
    assert second > first
    fbuild.build()
    assert os.stat(fbuild.BIND).st_mtime_ns == second
