"""When the operators' binding is rebuilt."""
import sys

import pytest
import torch

from bit_quantized_moe_top_b200 import build


@pytest.fixture
def built(monkeypatch):
    """The binding is there and current; further builds of it are only noted."""
    build.build()
    calls = []
    monkeypatch.setattr(build, "build_binding", lambda: calls.append(1))
    monkeypatch.setattr(build, "build_library", lambda *a: pytest.fail("the library is current"))
    return calls


def test_current_binding_is_kept(built):
    assert build.up_to_date()
    assert build.build() == build.LIB and not built


def test_binding_of_another_torch_is_rebuilt(built, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not build.up_to_date()
    build.build()
    assert built == [1]


def test_binding_of_another_python_is_rebuilt(built, monkeypatch):
    import sysconfig
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-000-other" if n == "SOABI" else real(n))
    assert not build.up_to_date()
    build.build()
    assert built == [1]


def test_library_without_torch(built, monkeypatch, tmp_path):
    """The C ABI needs nvcc alone: without torch there is no binding to build or to miss."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert build.up_to_date()
    assert build.build() == build.LIB and build.build(force=False) == build.LIB
    assert not built


def test_library_beside_a_torch_without_cuda(built, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(torch.version, "cuda", None)
    assert build.up_to_date() and build.build() == build.LIB and not built
