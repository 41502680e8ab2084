"""What the build needs (CPU)."""

import os
import subprocess
import sys

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "paged_kv_cache_51_gb300")

# _build.py run as a program by an interpreter that has no torch
WITHOUT_TORCH = """
import runpy, sys
sys.modules["torch"] = None
sys.argv = sys.argv[1:]
runpy.run_path(sys.argv[0], run_name="__main__")
"""


@pytest.mark.parametrize("args", [[], ["--library"]])
def test_the_library_is_built_without_torch(lib, args):
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH, os.path.join(PACKAGE, "_build.py")]
                       + args, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().endswith("libpagedkv.so")


def test_the_extension_is_left_out_on_request(lib, monkeypatch):
    from paged_kv_cache_51_gb300 import _build

    def needed(*args):
        raise AssertionError("the extension was compiled")

    monkeypatch.setattr(_build, "_compile_binding", needed)
    assert _build.build(binding=False) == _build.LIB
    with pytest.raises(AssertionError):
        _build.build()
