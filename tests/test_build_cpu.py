"""The build: what one part's failure leaves of the others."""
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
