"""The module that marshals a decode step's calls belongs to one Python and one torch, and can be missing (CPU)."""
import os
import sysconfig

import pytest
import torch

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec


def test_another_torch_or_python_has_another_module(monkeypatch):
    here = dec.calls_path()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert torch.__version__ in here and here.endswith(suffix)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0+other")
        assert dec.calls_path() != here
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        assert dec.calls_path() != here
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".other.so" if name == "EXT_SUFFIX" else None)
        assert dec.calls_path() != here
    assert dec.calls_path() == here


def test_what_was_built_for_another_torch_is_not_loaded(monkeypatch):
    tld_build.build()
    assert dec.load_calls() is not None
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert dec.load_calls() is None


def test_built_where_the_loader_looks():
    assert tld_build.build_calls() == dec.calls_path() and os.path.exists(dec.calls_path())


def test_without_torch_s_headers_the_library_is_built_all_the_same(monkeypatch, tmp_path):
    monkeypatch.setattr(torch, "__file__", str(tmp_path / "__init__.py"))
    with pytest.warns(RuntimeWarning, match="python_variable.h is missing"):
        assert tld_build.build_calls() is None
    with pytest.warns(RuntimeWarning):
        assert os.path.exists(tld_build.build())
