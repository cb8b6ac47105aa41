"""Calls of several sizes from several threads at once: each thread's calls succeed and give the bits that they give alone,
whatever sizes of the same kernels the other threads launch meanwhile.

The threads are native ones: Python's take turns, and hardly ever are two of them inside the library."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, U8, gen, randn, unwritten, workspace

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I, N = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    lib = tmp_path_factory.mktemp("threads") / "libmany_threads.so"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-pthread", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "native", "many_threads.cpp"), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def at_once(run, entry, calls, out, times):
    """Each of `calls` alone, then all of them at once on a thread and a stream of its own, `times` times each."""
    fn = ctypes.cast(getattr(coat.lib(), entry), P)
    run.restype, run.argtypes = I, [P, P, ctypes.c_int, I]
    one = type(calls[0]) * 1
    want = []
    for call, o in zip(calls, out):
        assert run(fn, one(call), 1, 1) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    assert run(fn, (type(calls[0]) * len(calls))(*calls), len(calls), times) == 0
    torch.cuda.synchronize()
    for o, ref in zip(out, want):
        assert all(torch.equal(a.view(U8), b.view(U8)) for a, b in zip(o, ref))


class EmbedCall(ctypes.Structure):
    _fields_ = [("dout", P), ("ids", P), ("M", I), ("V", I), ("C", I), ("dtable", P), ("workspace", P), ("bytes", N), ("stream", P)]


def test_embedding_gradients_of_several_tables(native):
    """The sorting kernel's shared memory goes by the table's rows: 4, 62 and 176 KB here."""
    M, C = 40, 16
    calls, out, keep = [], [], []
    for V in (2000, 32000, 90000):
        dout, ids = randn(M, C, seed=V).to(BF), torch.randint(-1, V, (M,), generator=gen(V), device="cuda")
        d, ws = unwritten(V, C), workspace(coat.coat_embedding_backward_workspace_bytes(M, V, C))
        stream = torch.cuda.Stream()
        keep += [dout, ids, ws, stream]
        calls.append(EmbedCall(dout.data_ptr(), ids.data_ptr(), M, V, C, d.data_ptr(), ws.data_ptr(), ws.numel(), stream.cuda_stream))
        out.append([d])
    torch.cuda.synchronize()
    at_once(native.embed_at_once, "coat_embedding_backward", calls, out, 5000)
    del keep


class NormCall(ctypes.Structure):
    _fields_ = [(n, P) for n in ("dy", "q", "scale", "rstd", "weight")] + [("M", I), ("N", I), ("dx", P), ("dweight", P),
                                                                            ("workspace", P), ("bytes", N), ("stream", P)]


def test_norm_gradients_of_several_widths(native):
    """The backward kernel's shared memory goes by the width: 52, 96 and 128 KB here, of the same kernel."""
    M, G = 20, 16
    calls, out, keep = [], [], []
    for width in (4096, 6144, 8192):
        x, w, dy = randn(M, width, seed=width).to(BF), torch.ones(width, device="cuda"), randn(M, width, seed=width + 1).to(BF)
        y, q = unwritten(M, width), unwritten(M, width, dtype=U8)
        scale, rstd = torch.empty(M, width // G, device="cuda"), torch.empty(M, device="cuda")
        coat.coat_rmsnorm_ckpt(x, w, 1e-5, G, y, q, scale, rstd)
        dx, dw = unwritten(M, width), unwritten(width)
        ws = workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, width))
        stream = torch.cuda.Stream()
        keep += [w, dy, q, scale, rstd, ws, stream]
        calls.append(NormCall(dy.data_ptr(), q.data_ptr(), scale.data_ptr(), rstd.data_ptr(), w.data_ptr(), M, width, dx.data_ptr(),
                              dw.data_ptr(), ws.data_ptr(), ws.numel(), stream.cuda_stream))
        out.append([dx, dw])
    torch.cuda.synchronize()
    at_once(native.norm_at_once, "coat_rmsnorm_ckpt_backward", calls, out, 5000)
    del keep
