"""Building the library where the Python binding of the paged calls cannot be built (CPU)."""
import os
import sys

import pytest

from compressed_kv_cache_gva_b200 import _build, gva


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    _build.build_bind()


def test_library_is_built_without_a_host_compiler(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "bind_path", lambda: str(tmp_path / "_bind.so"))
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    with pytest.warns(UserWarning, match="binding"):
        assert _build.build() == _build.LIB
    with pytest.raises(OSError):
        _build.build_bind()


def test_library_is_built_without_torch(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "bind_path", lambda: str(tmp_path / "_bind.so"))
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="binding"):
        assert _build.build() == _build.LIB
    with pytest.raises(ImportError):
        _build.build_bind()


def test_library_is_built_where_the_binding_does_not_compile(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "bind_path", lambda: str(tmp_path / "_bind.so"))
    monkeypatch.setenv("CXX", "false")
    with pytest.warns(UserWarning, match="binding"):
        assert _build.build() == _build.LIB
    assert os.path.exists(gva.LIB_PATH)


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    import torch
    here = _build.bind_path()
    assert os.path.exists(here)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert _build.bind_path() != here and not os.path.exists(_build.bind_path())
    monkeypatch.setattr(gva, "_bind", None)
    with pytest.raises(RuntimeError, match="missing: build it"):
        gva._paged()


def test_a_binding_of_another_python_is_not_loaded(monkeypatch):
    here = _build.bind_path()
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert _build.bind_path() != here
    monkeypatch.setattr(gva, "_bind", None)
    with pytest.raises(RuntimeError, match="missing: build it"):
        gva._paged()
