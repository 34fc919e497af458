"""The compiled binding is the cache operators' alone: what needs no device."""
import ctypes
import os

import pytest

from draft_selection_dflash2_gb300 import _lib, api, build


class FakeLibrary:
    def dflash2_create(self, device, handle):
        handle._obj.value = 64
        return 0

    def dflash2_destroy(self, handle):
        return 0


@pytest.fixture
def unloaded(monkeypatch):
    monkeypatch.setattr(_lib, "_bind", None)


def test_a_handle_needs_no_binding(monkeypatch, unloaded, tmp_path):
    monkeypatch.setattr(_lib, "load", lambda: FakeLibrary())
    monkeypatch.setattr(_lib, "BIND_PATH", str(tmp_path / "missing.so"))
    with api.Handle(0) as h:
        assert h.raw == 64 and isinstance(h.ptr, ctypes.c_void_p)
        with pytest.raises(RuntimeError, match="missing.so is missing"):
            h._bind


def test_the_library_is_built_without_a_host_compiler(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "bind.so"))
    with pytest.warns(UserWarning, match="cache operators"):
        assert os.path.exists(build.build())
    with pytest.raises(OSError):
        build.build_bind()
    assert not os.path.exists(build.BIND)


def test_a_binding_for_another_torch_is_refused(monkeypatch, unloaded, tmp_path):
    import torch
    build.build()
    assert _lib.load_bind().torch_version == torch.__version__
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch"):
        _lib.load_bind()
    broken = tmp_path / "broken.so"
    broken.write_bytes(b"no module")
    monkeypatch.setattr(_lib, "BIND_PATH", str(broken))
    with pytest.raises(RuntimeError, match="does not load"):
        _lib.load_bind()
