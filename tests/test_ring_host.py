"""Host-side check of ring.h, by which a block that stops early waits for its copies (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "coat_fp8_adamw_gb300", "csrc")


def test_a_block_that_stops_waits_for_every_copy_it_has_started(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "ring_check"
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "ring_check.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    stats = dict(kv.split("=") for kv in out.split())
    assert int(stats["cases"]) == 3 * 19 * 20 // 2 and int(stats["wrong"]) == 0
