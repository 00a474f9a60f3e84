"""What build() needs: the library is built without Python's headers, and the paged-cache calls then stay in Python."""
import os
import sys
import sysconfig

import pytest

from attention_forward_prefill_gb300 import binding, build


def test_a_host_without_python_headers_builds_the_library(monkeypatch, tmp_path, capfd):
    build.build()
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / "_paged_calls.so"))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert not os.path.exists(build.CALLS_PATH)
    assert "Python.h" in capfd.readouterr().err


def test_the_library_is_built_before_the_module(monkeypatch):
    order = []
    monkeypatch.setattr(build, "_build_library", lambda *a: order.append("library"))
    monkeypatch.setattr(build, "_build_calls", lambda *a: order.append("calls"))
    build.build(force=True)
    assert order == ["library", "calls"]


def test_calls_without_the_module_go_through_python(monkeypatch):
    torch = pytest.importorskip("torch")
    build.build()
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setitem(sys.modules, "attention_forward_prefill_gb300._paged_calls", None)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.decode_paged(torch.zeros(1, 2, 64, dtype=torch.float16), k, k, torch.zeros(1, 1, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32))
    assert binding._calls.decode() is NotImplemented
