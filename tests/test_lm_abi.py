"""What the embedding, its gradient and dropout refuse, through the C ABI and through the binding (CPU only: no call here
reaches a kernel; the addresses are made up)."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from coat_fp8_adamw_gb300 import _build

A = 1 << 20
STEP = 1 << 24


def at(i, off=0):
    return A + i * STEP + off


@pytest.fixture(scope="module")
def L():
    _build.build()
    return coat.lib()


def _emb(L, table=at(0), ids=at(1), wide=0, scale=1.0, M=64, V=100, C=64, out=at(2)):
    return L.coat_embedding(table, ids, wide, scale, M, V, C, out, None)


def test_embedding(L):
    assert _emb(L) == 5 and _emb(L, wide=1, M=1, V=1, C=16, scale=-0.5) == 5
    for k in ("table", "ids", "out"):
        assert _emb(L, **{k: 0}) == 1
    for k in ("M", "V", "C"):
        assert _emb(L, **{k: 0}) == 1 and _emb(L, **{k: -16}) == 1 and _emb(L, **{k: 1 << 31}) == 1
    assert _emb(L, C=72) == 1 and _emb(L, C=8) == 1
    assert _emb(L, M=(1 << 31) - 1, C=1 << 20) == 1                     # more elements than any entry point takes
    for s in (float("nan"), float("inf"), -float("inf")):
        assert _emb(L, scale=s) == 1
    assert _emb(L, table=at(0, 8)) == 2 and _emb(L, ids=at(1, 4)) == 2 and _emb(L, out=at(2, 2)) == 2
    assert _emb(L, out=at(0)) == 1 and _emb(L, out=at(0, 100 * 64 * 2 - 16)) == 1 and _emb(L, out=at(0, 100 * 64 * 2)) == 5
    assert _emb(L, ids=at(2, 16)) == 1
    assert _emb(L, ids=at(1), out=at(1, 4 * 64)) == 5 and _emb(L, wide=1, ids=at(1), out=at(1, 4 * 64)) == 1


def _emb_b(L, dout=at(0), ids=at(1), wide=0, scale=1.0, M=64, V=100, C=64, add=0, dtable=at(2), ws=at(3), n=1 << 20):
    return L.coat_embedding_backward(dout, ids, wide, scale, M, V, C, add, dtable, ws, n, None)


def test_embedding_backward(L):
    assert _emb_b(L) == 5 and _emb_b(L, add=1, wide=1) == 5
    for k in ("dout", "ids", "dtable", "ws"):
        assert _emb_b(L, **{k: 0}) == 1
    for k in ("M", "V", "C"):
        assert _emb_b(L, **{k: 0}) == 1
    assert _emb_b(L, C=24) == 1 and _emb_b(L, scale=float("nan")) == 1
    assert _emb_b(L, dtable=at(2, 8)) == 2 and _emb_b(L, ws=at(3, 8)) == 2
    assert _emb_b(L, dtable=at(0)) == 1 and _emb_b(L, ws=at(2)) == 1 and _emb_b(L, ws=at(1)) == 1


def test_embedding_backward_workspace(L):
    f = L.coat_embedding_backward_workspace_bytes
    # eight bytes a token, in multiples of 16; two float32 rows for every chunk of 32; a flag for 128 k >= V rows
    assert f(1, 1, 16) == 16 + 128 + 128 and f(3, 129, 16) == 32 + 128 + 256
    assert f(32, 128, 16) == 256 + 128 + 128 and f(63, 1, 64) == 512 + 1024 + 128
    assert f(0, 1, 16) == 0 and f(16, 1, 24) == 0 and f(1 << 31, 1, 16) == 0 and f(16, 0, 16) == 0


def _drop(L, x=at(0), res=None, p=0.1, rng=at(1), n=1000, y=at(2)):
    return L.coat_dropout(x, res, p, rng, n, y, None)


def test_dropout(L):
    assert _drop(L) == 5 and _drop(L, res=at(3)) == 5 and _drop(L, n=1) == 5 and _drop(L, p=0.0) == 5
    for k in ("x", "rng", "y"):
        assert _drop(L, **{k: 0}) == 1
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 65535.5 / 65536):
        assert _drop(L, p=p) == 1
    assert _drop(L, p=65535.25 / 65536) == 5
    assert _drop(L, n=0) == 1 and _drop(L, n=-1) == 1 and _drop(L, n=coat.MAX_N + 1) == 1
    assert _drop(L, x=at(0, 2)) == 2 and _drop(L, rng=at(1, 8)) == 2 and _drop(L, res=at(3, 8)) == 2
    assert _drop(L, y=at(0)) == 1 and _drop(L, y=at(1)) == 1 and _drop(L, res=at(2)) == 1
    assert _drop(L, y=at(0, 2000)) == 5


def test_dropout_backward(L):
    def back(dy=at(0), p=0.1, rng=at(1), n=1000, dx=at(2)):
        return L.coat_dropout_backward(dy, p, rng, n, dx, None)
    assert back() == 5
    assert back(dy=0) == 1 and back(rng=0) == 1 and back(dx=0) == 1 and back(p=1.0) == 1 and back(n=0) == 1
    assert back(dx=at(0, 16)) == 1 and back(dx=at(2, 8)) == 2


def test_binding_refuses_what_is_not_on_a_gpu():
    table, out = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.bfloat16)
    ids, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        coat.coat_embedding(table, ids, 1.0, out)
    with pytest.raises(ValueError, match="CUDA"):
        coat.coat_embedding_backward(out, ids, 1.0, table, ws)
    with pytest.raises(ValueError, match="CUDA"):
        coat.coat_dropout(table, 0.1, rng, table.clone())
    with pytest.raises(ValueError, match="CUDA"):
        coat.coat_dropout_backward(table, 0.1, rng, table.clone())
    with pytest.raises(ValueError, match="2-D"):
        coat.coat_embedding(table.flatten(), ids, 1.0, out)
    with pytest.raises(TypeError, match="int32"):
        coat.coat_embedding(table, ids.float(), 1.0, out)


def _lce(L, x=at(0), ld=64, w=at(1), t=at(2), wide=0, M=64, V=100, C=64, loss=at(3), lse=at(4), ws=at(5), n=1 << 20):
    return L.coat_linear_cross_entropy(x, ld, w, t, wide, M, V, C, loss, lse, ws, n, None)


def test_linear_cross_entropy(L):
    assert _lce(L) == 5 and _lce(L, wide=1, ld=72, V=1, M=1) == 5
    for k in ("x", "w", "t", "loss", "lse", "ws"):
        assert _lce(L, **{k: 0}) == 1
    for k in ("M", "V", "C"):
        assert _lce(L, **{k: 0}) == 1 and _lce(L, **{k: 1 << 31}) == 1
    assert _lce(L, C=24, ld=24) == 1 and _lce(L, ld=56) == 1 and _lce(L, ld=68) == 1
    assert _lce(L, M=1 << 20, V=(1 << 20) + 1, C=16, ld=16) == 1        # more logits than any entry point takes elements
    assert _lce(L, x=at(0, 8)) == 2 and _lce(L, lse=at(4, 4)) == 2
    assert _lce(L, loss=at(0)) == 1 and _lce(L, lse=at(3)) == 1 and _lce(L, ws=at(4)) == 1 and _lce(L, ws=at(1)) == 1


def _lce_b(L, x=at(0), ld=64, w=at(1), t=at(2), wide=0, lse=at(3), g=at(4), h=None, M=64, V=1000, C=64, piece=0, dx=at(5), dw=at(6),
           ws=at(7), n=1 << 20):
    return L.coat_linear_cross_entropy_backward(x, ld, w, t, wide, lse, g, h, M, V, C, piece, dx, dw, ws, n, None)


def test_linear_cross_entropy_backward(L):
    assert _lce_b(L) == 5 and _lce_b(L, h=at(8), wide=1) == 5 and _lce_b(L, piece=300) == 5
    for k in ("x", "w", "t", "lse", "g", "dx", "dw", "ws"):
        assert _lce_b(L, **{k: 0}) == 1
    for k in ("M", "V", "C"):
        assert _lce_b(L, **{k: 0}) == 1
    assert _lce_b(L, piece=-1) == 1 and _lce_b(L, ld=60) == 1 and _lce_b(L, h=at(8, 8)) == 2
    assert _lce_b(L, piece=(1 << 63) - 1) == 5
    assert _lce_b(L, dx=at(0)) == 1 and _lce_b(L, dw=at(1)) == 1 and _lce_b(L, dx=at(6)) == 1 and _lce_b(L, h=at(6)) == 1


def test_linear_cross_entropy_workspaces(L):
    f, b = L.coat_linear_cross_entropy_workspace_bytes, L.coat_linear_cross_entropy_backward_workspace_bytes
    assert f(0, 10) == 0 and f(1 << 20, (1 << 20) + 1) == 0 and f(1, 1) > 0
    assert b(10, 100, 24, 0) == 0 and b(10, 100, 64, -1) == 0
    xt = 2 * 64 * 16 + 16                                                # x transposed, its rows in multiples of eight, and a factor
    assert b(10, 100, 64, 0) == b(10, 100, 64, 1) == b(10, 100, 64, (1 << 63) - 1) == 2 * 10 * 256 + xt    # one piece
    assert b(10, 1000, 64, 300) == 2 * 10 * 512 + xt + 4 * 10 * 64       # two: and dx's sums between them
    M, V, C = 8192, 32000, 4096
    assert b(M, V, C, 0) == 2 * M * V + 2 * M * C + 16                         # one piece: its dz is within 512 MiB
    M = 16384                                                             # two of about the same width
    assert b(M, V, C, 0) == 2 * M * 16128 + 2 * M * C + 16 + 4 * M * C and 2 * M * 16128 <= 512 << 20
