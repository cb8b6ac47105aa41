"""Host-side check of divide.h, by which the gated unit finds an element's row (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "coat_fp8_adamw_gb300", "csrc")


def test_the_multiplication_is_the_division(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "divide_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "divide_check.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    stats = dict(kv.split("=") for kv in out.split())
    assert int(stats["cases"]) > 2 * 10 ** 8 and int(stats["wrong"]) == 0
