"""The extension of the paged calls is rebuilt for another PyTorch or Python, and nothing else needs it."""
import sysconfig

import pytest
import torch

from quantized_kv_cache_kv8_gb300 import build


@pytest.fixture(autouse=True)
def built():
    build.build()
    assert build.up_to_date()


def test_another_pytorch_rebuilds_the_extension(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.up_to_date()


def test_another_python_rebuilds_the_extension(monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda k: ".other.so" if k == "EXT_SUFFIX" else real(k))
    assert not build.up_to_date()


def test_the_library_needs_no_cxx_compiler(monkeypatch, tmp_path):
    """Without a compiler for the extension the kernels are built and found; the extension says what is missing."""
    monkeypatch.setattr(build, "HOST", str(tmp_path / "host.so"))
    monkeypatch.setattr(build, "HOST_STAMP", str(tmp_path / "host.stamp"))
    monkeypatch.setenv("CXX", str(tmp_path / "no-compiler"))
    assert build.build_library() == build.LIB
    with pytest.raises(RuntimeError, match="no-compiler"):
        build.build_host()
    with pytest.raises(RuntimeError, match="no-compiler"):
        build.build()


def test_a_new_extension_leaves_a_stamp(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "HOST", str(tmp_path / "host.so"))
    monkeypatch.setattr(build, "HOST_STAMP", str(tmp_path / "host.stamp"))
    assert not build.host_up_to_date()
    build.build_host()
    assert build.host_up_to_date()
    (tmp_path / "host.stamp").write_text("torch 0.0.1\n")
    assert not build.host_up_to_date()
