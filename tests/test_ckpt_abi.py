"""What the checkpointing operators refuse, through the C ABI (CPU only: no call
here reaches a kernel; the addresses are made up)."""
import pytest

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


def _norm(L, x=at(0), res=None, w=at(1), eps=1e-5, M=64, N=256, G=128, h=None, y=at(2), q=at(3), S=at(4), r=at(5)):
    return L.coat_rmsnorm_ckpt(x, res, w, eps, M, N, G, h, y, q, S, r, None)


def test_norm_forward(L):
    assert _norm(L) == 5                                   # well formed, but not device memory
    assert _norm(L, res=at(6), h=at(7)) == 5
    for k in ("x", "w", "y", "q", "S", "r"):
        assert _norm(L, **{k: 0}) == 1
    assert _norm(L, res=at(6)) == 1 and _norm(L, h=at(7)) == 1   # a residual and h come together
    assert _norm(L, M=0) == 1 and _norm(L, M=1 << 31) == 1
    assert _norm(L, N=0) == 1 and _norm(L, N=16384 + 128) == 1 and _norm(L, N=16384) == 5
    assert _norm(L, N=264, G=8) == 1 and _norm(L, N=272, G=16) == 5 and _norm(L, N=272, G=32) == 1
    for G in (0, 4, 24, 256, -8):
        assert _norm(L, G=G) == 3
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _norm(L, eps=eps) == 1
    assert _norm(L, x=at(0, 8)) == 2 and _norm(L, r=at(5, 4)) == 2
    assert _norm(L, y=at(0, 64 * 256 * 2 - 16)) == 1       # y overlaps x
    assert _norm(L, y=at(0, 64 * 256 * 2)) == 5            # and just does not
    assert _norm(L, q=at(2, 16)) == 1 and _norm(L, r=at(4)) == 1


def _norm_b(L, dy=at(0), q=at(1), S=at(2), r=at(3), w=at(4), dres=None, M=64, N=256, G=64, dx=at(5), dw=at(6), ws=at(7),
            n=1 << 20):
    return L.coat_rmsnorm_ckpt_backward(dy, q, S, r, w, dres, M, N, G, dx, dw, ws, n, None)


def test_norm_backward(L):
    assert _norm_b(L) == 5 and _norm_b(L, dres=at(8)) == 5
    for k in ("dy", "q", "S", "r", "w", "dx", "dw", "ws"):
        assert _norm_b(L, **{k: 0}) == 1
    assert _norm_b(L, G=12) == 3 and _norm_b(L, N=288) == 1 and _norm_b(L, M=-1) == 1
    assert _norm_b(L, ws=at(7, 8)) == 2 and _norm_b(L, dres=at(8, 2)) == 2
    assert _norm_b(L, dx=at(0)) == 1 and _norm_b(L, dw=at(7, 16)) == 1 and _norm_b(L, dx=at(1)) == 1
    assert L.coat_rmsnorm_ckpt_backward_workspace_bytes(0, 256) == 0
    assert L.coat_rmsnorm_ckpt_backward_workspace_bytes(64, 1 << 20) == 0


def _sw(L, g=at(0), u=at(1), ld=256, M=64, N=256, G=128, h=at(2), gq=at(3), gs=at(4), uq=at(5), us=at(6)):
    return L.coat_swiglu_ckpt(g, u, ld, M, N, G, h, gq, gs, uq, us, None)


def test_swiglu_forward(L):
    assert _sw(L) == 5
    assert _sw(L, u=at(0, 512), ld=512) == 5                # halves of one tensor
    for k in ("g", "u", "h", "gq", "gs", "uq", "us"):
        assert _sw(L, **{k: 0}) == 1
    assert _sw(L, ld=248) == 1 and _sw(L, ld=260) == 1 and _sw(L, ld=264) == 5
    assert _sw(L, G=129) == 3 and _sw(L, N=136, G=8) == 1
    assert _sw(L, u=at(1, 2)) == 2
    assert _sw(L, h=at(0)) == 1 and _sw(L, uq=at(3)) == 1


def _sw_b(L, dh=at(0), gq=at(1), gs=at(2), uq=at(3), us=at(4), M=64, N=256, G=128, dg=at(5), du=at(6), ld=256, hq=None, hs=None):
    return L.coat_swiglu_ckpt_backward(dh, gq, gs, uq, us, M, N, G, dg, du, ld, hq, hs, None)


def test_swiglu_backward(L):
    assert _sw_b(L) == 5 and _sw_b(L, hq=at(7), hs=at(8)) == 5
    assert _sw_b(L, du=at(5, 512), ld=512) == 5             # halves of one tensor
    assert _sw_b(L, dg=at(6, 512), ld=512) == 5             # in either order
    assert _sw_b(L, du=at(5, 496), ld=512) == 1             # ranges that meet
    assert _sw_b(L, du=at(5, 528), ld=512) == 1             # the end of a row meets the next one
    assert _sw_b(L, du=at(5)) == 1
    assert _sw_b(L, hq=at(7)) == 1 and _sw_b(L, hs=at(8)) == 1
    for k in ("dh", "gq", "gs", "uq", "us", "dg", "du"):
        assert _sw_b(L, **{k: 0}) == 1
    assert _sw_b(L, dg=at(0)) == 1 and _sw_b(L, du=at(3)) == 1 and _sw_b(L, hq=at(6), hs=at(8)) == 1
    assert _sw_b(L, G=4) == 3 and _sw_b(L, du=at(6, 8)) == 2


def _qk(L, q=at(0), q_ld=512, Hq=4, k=at(1), k_ld=256, Hk=2, D=128, qw=at(2), kw=at(3), eps=1e-5, c=at(4), s=at(5), mp=64,
        rot=128, pos=at(6), M=16, G=64, qo=at(7), qq=at(8), qs=at(9), qr=at(10), ko=at(11), kq=at(12), ks=at(13), kr=at(14)):
    return L.coat_qk_norm_rope_ckpt(q, q_ld, Hq, k, k_ld, Hk, D, qw, kw, eps, c, s, mp, rot, pos, 0, M, G, qo, qq, qs, qr,
                                    ko, kq, ks, kr, None)


def test_qk_forward(L):
    assert _qk(L) == 5
    for n in ("q", "k", "qw", "kw", "c", "s", "pos", "qo", "qq", "qs", "qr", "ko", "kq", "ks", "kr"):
        assert _qk(L, **{n: 0}) == 1
    none = dict(k=0, kw=0, ko=0, kq=0, ks=0, kr=0)
    assert _qk(L, Hk=0, **none) == 5                         # queries alone
    assert _qk(L, Hk=0, Hq=0, **none) == 1
    assert _qk(L, Hk=-1, **none) == 1
    assert _qk(L, k=at(0, 1024), q_ld=1024, k_ld=1024) == 5  # ranges of one projection
    assert _qk(L, D=8) == 1 and _qk(L, D=264, G=8) == 1 and _qk(L, D=120, G=8) == 1 and _qk(L, D=96, rot=96) == 1
    assert _qk(L, rot=0) == 1 and _qk(L, rot=24) == 1 and _qk(L, rot=144) == 1 and _qk(L, rot=64) == 5
    assert _qk(L, G=256) == 3 and _qk(L, mp=0) == 1 and _qk(L, M=0) == 1 and _qk(L, eps=0.0) == 1
    assert _qk(L, q_ld=504) == 1 and _qk(L, k_ld=260) == 1
    assert _qk(L, pos=at(6, 4)) == 2
    assert _qk(L, qo=at(1)) == 1 and _qk(L, kr=at(10)) == 1


def _qk_b(L, dqo=at(0), dko=at(1), qq=at(2), qs=at(3), qr=at(4), kq=at(5), ks=at(6), kr=at(7), Hq=4, Hk=2, D=128, qw=at(8),
          kw=at(9), c=at(10), s=at(11), mp=64, rot=128, pos=at(12), M=16, G=64, dq=at(13), dq_ld=512, dk=at(14), dk_ld=256,
          dqw=at(15), dkw=at(16), ws=at(17), n=1 << 20):
    return L.coat_qk_norm_rope_ckpt_backward(dqo, dko, qq, qs, qr, kq, ks, kr, Hq, Hk, D, qw, kw, c, s, mp, rot, pos, 0, M, G,
                                             dq, dq_ld, dk, dk_ld, dqw, dkw, ws, n, None)


def test_qk_backward(L):
    assert _qk_b(L) == 5
    for n in ("dqo", "dko", "qq", "qs", "qr", "kq", "ks", "kr", "qw", "kw", "c", "s", "pos", "dq", "dk", "dqw", "dkw", "ws"):
        assert _qk_b(L, **{n: 0}) == 1
    assert _qk_b(L, dk=at(13, 1024), dq_ld=768, dk_ld=768) == 5   # ranges of one gradient buffer
    assert _qk_b(L, dk=at(13, 1024), dq_ld=760, dk_ld=760) == 1   # that meet
    assert _qk_b(L, dk=at(13, 1024), dq_ld=768, dk_ld=1024) == 1  # strides that differ
    assert _qk_b(L, dq=at(0)) == 1 and _qk_b(L, dkw=at(15)) == 1
    assert _qk_b(L, G=16, D=80, rot=80, dq_ld=320, dk_ld=160) == 5
    assert _qk_b(L, dk=at(14, 8)) == 2
    assert L.coat_qk_norm_rope_ckpt_backward_workspace_bytes(16, 24) == 0


def _wg(L, dy=at(0), ld=512, q=at(1), S=at(2), r=None, c=None, M=64, N=512, K=256, G=64, dw=at(3), ws=at(4), n=1 << 20):
    return L.coat_ckpt_weight_grad(dy, ld, q, S, r, c, M, N, K, G, dw, ws, n, None)


def test_weight_gradient(L):
    assert _wg(L) == 5 and _wg(L, r=at(5), c=at(6)) == 5
    for k in ("dy", "q", "S", "dw", "ws"):
        assert _wg(L, **{k: 0}) == 1
    assert _wg(L, M=0) == 1 and _wg(L, N=516, ld=520) == 1 and _wg(L, K=264, G=8) == 1 and _wg(L, K=288) == 1
    assert _wg(L, ld=504) == 1 and _wg(L, ld=520) == 5 and _wg(L, N=520, ld=520) == 5
    assert _wg(L, G=2) == 3 and _wg(L, r=at(5, 4)) == 2
    assert _wg(L, dw=at(0)) == 1 and _wg(L, ws=at(3)) == 1 and _wg(L, c=at(3)) == 1
    assert L.coat_ckpt_weight_grad_workspace_bytes(64, 0, 16) == 0
