"""The build of the module that marshals the int8 calls: one for each interpreter, and none without its headers."""

import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from paged_kv_cache_111_gb300 import _build


@pytest.fixture(autouse=True, scope="module")
def built():
    _build.build()


def test_the_module_carries_the_interpreters_tag(monkeypatch):
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(_build.CALLS) == "_py_calls" + tag and len(tag) > len(".so")
    assert _build.up_to_date()
    # another interpreter's is not this one's
    monkeypatch.setattr(_build, "CALLS", _build.CALLS.replace(tag, ".cpython-30-other.so"))
    assert not _build.up_to_date()


def test_a_compiler_with_arguments(monkeypatch, tmp_path):
    monkeypatch.setenv("CC", "gcc -pipe -DNDEBUG")
    out = str(tmp_path / os.path.basename(_build.CALLS))
    _build.build_calls(out)
    assert os.path.getsize(out) > 1000
    monkeypatch.setenv("CC", "gcc --no-such-flag")
    with pytest.raises(RuntimeError, match="py_calls.c failed"):
        _build.build_calls(out)


def test_without_headers(monkeypatch, tmp_path, capsys):
    """The int8 calls say what is missing, the others do not need it."""
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    missing = str(tmp_path / "_py_calls.so")
    monkeypatch.setattr(_build, "CALLS", missing)
    monkeypatch.setattr(pkv, "_module", None)
    _build.build_calls(missing)
    assert not os.path.exists(missing) and "Python.h" in capsys.readouterr().err
    assert _build.up_to_date()
    x = torch.zeros(3, 2, 64)
    with pytest.raises(RuntimeError, match="build it first"):
        pkv.copy_blocks_int8(x, x, x)
    with pytest.raises(ValueError, match="CUDA tensors"):
        pkv.paged_attn_combine(x, x)


def test_the_package_imports_the_tagged_module_only():
    code = ("import paged_kv_cache_111_gb300 as pkv; from paged_kv_cache_111_gb300 import _build; "
            "assert pkv._calls().__file__ == _build.CALLS")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
