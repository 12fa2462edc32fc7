"""The build where the Python binding's marshalling module cannot be made: the library alone, as C callers need it."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

if not shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")):
    pytest.skip("needs hipcc", allow_module_level=True)

BUILD = """
import os, sys
{before}
from block_scaled_quantized_amd import build as b
b.BUILD, b.LIB, b.MARSHAL, b.SOURCES = {tmp!r}, os.path.join({tmp!r}, "libmxgemm.so"), os.path.join({tmp!r}, "_marshal.so"), ["page_pool.cpp"]
open(b.MARSHAL, "w").close()                     # of an earlier build: it would not fit the new library
b.build(verbose=True)
print("library", os.path.getsize(b.LIB) > 0, "module", os.path.exists(b.MARSHAL))
"""


@pytest.mark.parametrize("before,why", [("sys.modules['torch'] = None", "torch"),
                                        ("import shutil; shutil.which = lambda name, **kw: None", "g++"),
                                        ("import sysconfig; sysconfig.get_paths = lambda *a: {'include': '/nowhere'}", "Python.h")])
def test_build_without_what_the_binding_needs(tmp_path, before, why):
    r = subprocess.run([sys.executable, "-c", BUILD.format(before=before, tmp=str(tmp_path))], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "library True module False" in r.stdout
    assert "_marshal.so is not built" in r.stdout and why in r.stdout, r.stdout


def test_missing_module_says_what_to_do():
    code = ("import sys; sys.modules['block_scaled_quantized_amd._marshal'] = None\nfrom block_scaled_quantized_amd import api\n"
            "try:\n    api.mxkv_copy_run([], None)\nexcept ImportError as e:\n    print(e)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "python -m block_scaled_quantized_amd.build" in r.stdout, (r.stdout, r.stderr)
