"""Static shared memory of every kernel, as the assembler counts it: at most the 48 KB that the programming model gives a
block without asking (CPU only)."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from coat_fp8_adamw_gb300 import _build

LIMIT = 48 << 10


def _kernels(src):
    """(kernel, bytes of static shared memory) of a source file."""
    cmd = [_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-Xptxas=-v", "-I", _build.INCLUDE, "-I", _build.CSRC, "-c",
           os.path.join(_build.CSRC, src), "-o", os.devnull]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    name, found = None, []
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        name = m.group(1) if m else name
        if "Used" in line and name:
            m = re.search(r"(\d+) bytes smem", line)
            found.append((name, int(m.group(1)) if m else 0))
            name = None
    return found


def test_no_kernel_has_more_static_shared_memory_than_a_block_has():
    try:
        _build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not found")
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        kernels = [k for found in ex.map(_kernels, _build.SOURCES) for k in found]
    assert len(kernels) > 50
    over = [(n, b) for n, b in kernels if b > LIMIT]
    assert not over, over
