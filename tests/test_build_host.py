"""What _build builds, and which extension module is loaded (host only; nothing is
compiled)."""
import importlib.util
import os

import pytest
import torch

import split_kv_merge_attn_b200 as skv
from split_kv_merge_attn_b200 import _build


@pytest.fixture
def built(monkeypatch):
    """Names of what build() would compile."""
    names = []
    monkeypatch.setattr(_build, "_run", lambda cmd, name, verbose: names.append(name))
    return names


def test_the_module_of_another_pytorch_is_not_used(monkeypatch, built):
    here = _build.torch_lib()
    assert os.path.exists(here)
    monkeypatch.setattr(os.path, "getmtime", lambda path: 0.0)
    _build.build()
    assert built == []  # nothing is newer than what is there
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu999")
    assert _build.torch_lib() != here and not os.path.exists(_build.torch_lib())
    _build.build()
    assert built == [os.path.basename(_build.torch_lib())]
    with pytest.raises(RuntimeError, match="9.9.9.*is missing"):
        skv._torch_calls.__wrapped__()


def test_another_python_has_a_module_of_its_own(monkeypatch):
    here = _build.torch_lib()
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: ".cpython-999-x86_64-linux-gnu.so")
    assert _build.torch_lib() != here


def test_the_library_is_built_without_pytorch(monkeypatch, built):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(_build, "torch_lib", lambda: pytest.fail("there is no PyTorch"))
    assert _build.build(force=True) == _build.LIB
    assert built == ["libsplitkv.so"]
