"""What the in-tree build asks of the machine (compilers are not run)."""
import subprocess
import sys

import pytest


def test_the_library_needs_no_torch():
    code = """
import subprocess, sys
sys.modules["torch"] = None  # as where it is not installed
from fp4_sparse_attention_pack_b200 import _build
calls = []
subprocess.check_call = lambda cmd, **kw: calls.append(cmd[0])
assert _build.build(force=True) == _build.LIB
print(calls)
"""
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True).stdout
    assert got.strip() == "['nvcc']"


def test_the_module_of_calls_is_built_for_each_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    from fp4_sparse_attention_pack_b200 import _build
    calls = []
    monkeypatch.setattr(_build.subprocess, "check_call", lambda cmd, **kw: calls.append(cmd))
    here = _build.bind_path()
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    assert _build.bind_path() != here
    _build._build_bind(False)
    assert len(calls) == 1 and calls[0][0] == "g++" and _build.bind_path() in calls[0]
