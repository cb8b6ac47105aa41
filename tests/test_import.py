"""Importing the package does not import torch: the C ABI by ctypes, the version and the build need none of it (CPU only)."""
import subprocess
import sys
import pathlib

ROOT = str(pathlib.Path(__file__).resolve().parents[1])


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


def test_the_package_is_imported_without_torch():
    out = _run("import sys, coat_fp8_adamw_gb300 as c; print('torch' in sys.modules, len(c.EXPORTS) > 0, "
               "'coat_rmsnorm_ckpt' in dir(c), hasattr(c, 'no_such_name'), 'torch' in sys.modules)")
    assert out == ["False", "True", "True", "False", "False"]


def test_it_imports_where_there_is_no_torch():
    out = _run("import sys; sys.modules['torch'] = None\n"
               "import coat_fp8_adamw_gb300 as c\n"
               "print(c.num_groups(129, 128))\n"
               "try: c.coat_ckpt_weight_grad\n"
               "except ImportError: print('ImportError')")
    assert out == ["2", "ImportError"]


def test_every_public_name_is_there():
    out = _run("import coat_fp8_adamw_gb300 as c\n"
               "from coat_fp8_adamw_gb300 import *\n"
               "missing = [n for n in c.__all__ if n not in globals() or not hasattr(c, n)]\n"
               "print(len(missing), callable(coat_swiglu_ckpt), c.coat_swiglu_ckpt is c.ckpt.coat_swiglu_ckpt, "
               "c.coat_swiglu_ckpt is coat_swiglu_ckpt)")
    assert out == ["0", "True", "True", "True"]
    assert _run("import coat_fp8_adamw_gb300 as c; print(c.ckpt.__name__)") == ["coat_fp8_adamw_gb300.ckpt"]
