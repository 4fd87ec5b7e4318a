"""What building needs: libcat.so only nvcc, the marshalling module of the
operator plans torch and a C++ compiler as well."""
import os
import sys

import pytest

from fft_circulant_attention_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_the_library_builds_without_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="marshalling"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)


@pytest.mark.parametrize("cxx", ["/bin/false", "/no/such/compiler"])
def test_the_library_builds_without_a_compiler_for_the_module(monkeypatch, tmp_path, cxx):
    path = str(tmp_path / "_marshal.so")
    monkeypatch.setattr(build, "marshal_path", lambda: path)
    monkeypatch.setenv("CXX", cxx)
    with pytest.warns(RuntimeWarning, match="marshalling"):
        assert build.build() == build.LIB
    # A module of an earlier source is not left to be loaded.
    with open(path, "w"):
        pass
    os.utime(path, (0, 0))
    with pytest.warns(RuntimeWarning, match="marshalling"):
        build.build()
    assert not os.path.exists(path)


def test_the_plans_say_what_is_missing(monkeypatch, tmp_path):
    import fft_circulant_attention_gb300 as cat
    monkeypatch.setattr(build, "marshal_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(cat, "_MARSHAL", None)
    with pytest.raises(RuntimeError, match="build it with"):
        cat._marshal()
