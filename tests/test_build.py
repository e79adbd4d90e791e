"""The build of the library and of the extension module beside it (no GPU)."""
import os
import sysconfig

import pytest
import torch

from sparse_moe_layer_bias_gb300 import build


def test_the_library_is_built_where_the_extension_module_cannot_be(monkeypatch):
    """The C ABI needs neither g++ for the module nor the headers of torch and Python: a warning, and the library's path."""
    def fails(force=False):
        raise RuntimeError("no headers")
    build.build()
    monkeypatch.setattr(build, "build_calls", fails)
    with pytest.warns(UserWarning, match="no headers"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)


def test_the_module_says_which_compiler_is_missing(monkeypatch):
    monkeypatch.setenv("PATH", "")
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build.build_calls(force=True)


def test_the_modules_name_carries_what_it_was_built_against():
    name = os.path.basename(build.calls_path())
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert "cpython" in name
