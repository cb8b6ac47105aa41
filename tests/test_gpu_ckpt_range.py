"""Norms of finite rows and heads whose squares leave float32's range: 1/rms, the output and the gradients are those
of the formulas, in the whole range of bf16.  Forms and bounds as in test_gpu_ckpt.py; 1/rms of rows from 2^126 on is
a subnormal number, whose last bit, 2^-149, is at most 2^-21 of it: within the same 2^-19."""
import pytest
import torch

import _ckpt_ref as R
import coat_fp8_adamw_gb300 as coat
from test_gpu_ckpt import (BF, E, EPS, F32, U8, bf16_bound, check_checkpoint, checkpoint, empty, gen, grads, near, norm_w,
                           rope_tables, workspace)
from test_gpu_ckpt import _built  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu
# largest elements of the rows: around the root of float32's range (2^64 / sqrt(N) and 2^64), to the end of bf16's
POWERS = (0, 56, 57, 58, 60, 63, 64, 65, 80, 100, 120, 126, 127)


def far_rows(M, N, seed):
    """Rows that end at 2^p, p from POWERS in turn, ordinary ones between them; in every fourth a single large element."""
    x = torch.rand(M, N, generator=gen(seed), device="cuda", dtype=torch.float64) * 2 - 1
    p = torch.tensor(POWERS, device="cuda", dtype=torch.float64)[torch.arange(M, device="cuda") % len(POWERS)]
    x = x * torch.exp2(p)[:, None]
    alone = torch.arange(M, device="cuda") % 4 == 3
    x[alone] *= 2.0 ** -60
    x[alone, N // 2 + 1] = -torch.exp2(p[alone])
    return x.to(BF)


def check_norm(x, w, eps, y, q, S, rstd, G, what):
    ref, rr = R.rmsnorm(x.double(), w.double(), eps)
    near(rstd, rr, 2.0 ** -19 * rr, what + "rstd")
    near(y, ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), what + "y")
    check_checkpoint(q, S, x, G, what)


# one team of a warp and more per block, teams of several warps, one team per block up to 32 warps
@pytest.mark.parametrize("N,G", [(16, 8), (256, 128), (528, 16), (1024, 32), (4096, 128), (8208, 8), (12288, 64), (16384, 128)])
@pytest.mark.parametrize("res", [False, True])
def test_norm(N, G, res):
    M = 2 * len(POWERS) + 1
    x, w = far_rows(M, N, N), norm_w(N, 1)
    r = (x.double() * -0.5).to(BF) if res else None
    h = empty(M, N) if res else None
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, rstd, residual=r, h=h)
    src = (x.float() + r.float()).to(BF) if res else x
    if res:
        assert torch.equal(h, src)
    check_norm(src, w, EPS, y, q, S, rstd, G, f"{N} ")
    # and backward, from what the forward pass left
    dy, dx, dw = grads(M, N, 5), empty(M, N), empty(N)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw, workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N)))
    xv = checkpoint(src, G)[2]
    rx, rw, sx, sw = R.rmsnorm_backward(dy.double(), xv, rstd.double(), w.double())
    near(dx, rx, bf16_bound(rx) + 2.0 ** -18 * sx, "dx")
    near(dw, rw, bf16_bound(rw) + (M + 64) * E * sw, "dweight")


@pytest.mark.parametrize("eps", [1e-40, 1e38, 3e38])
def test_norm_with_any_eps(eps):
    """Also where it is eps, or the sum of the two, that leaves the range."""
    eps = float(torch.tensor(eps, dtype=F32))
    M, N, G = 3 * len(POWERS), 512, 32
    x, w = far_rows(M, N, 9), norm_w(N, 2)
    x[:13] = torch.full((13, N), 1.5 * 2.0 ** 63, device="cuda").to(BF)         # a mean square of 2^127.2
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, eps, G, y, q, S, rstd)
    check_norm(x, w, eps, y, q, S, rstd, G, "")


@pytest.mark.parametrize("D,rot,G,inter", [(16, 16, 16, False), (48, 32, 8, False), (64, 64, 64, True), (128, 128, 128, False),
                                           (112, 96, 16, False), (256, 64, 32, True), (256, 256, 128, False)])
def test_heads(D, rot, G, inter):
    """Large heads beside ordinary ones in the same warp."""
    M, H = 9, 7
    x, w = far_rows(M * H, D, D).view(M, H, D), 4 * norm_w(D, 3)       # a weight times an element may leave the range
    cos, sin = rope_tables(M, rot)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    y, q, S, rstd = empty(M, H, D), empty(M, H, D, dtype=U8), empty(M, H, D // G, dtype=F32), empty(M, H, dtype=F32)
    coat.coat_qk_norm_rope_ckpt(x, None, w, None, EPS, cos, sin, pos, G, y, q, S, rstd, interleaved=inter)
    c, s = cos.double(), sin.double()
    ref, rr = R.qk(x.double(), w.double(), EPS, c, s, rot, inter)
    size = R.rmsnorm(x.double(), w.double(), EPS)[0].abs()
    size = R.rotate(size, c.abs(), -s.abs(), rot, inter).abs() + R.rotate(size, c.abs(), s.abs(), rot, inter).abs()
    near(rstd, rr, 2.0 ** -19 * rr, "rstd")
    near(y, ref, bf16_bound(ref) + 2.0 ** -18 * size, "out")
    check_checkpoint(q, S, x, G, "heads")
    dy, dx, dw = grads(M, H * D, 5).view(M, H, D), empty(M, H, D), empty(D)
    ws = workspace(coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, D))
    coat.coat_qk_norm_rope_ckpt_backward(dy, None, q, S, rstd, None, None, None, w, None, cos, sin, pos, G, dx, None, dw, None,
                                         ws, interleaved=inter)
    xv = checkpoint(x, G)[2]
    D64 = dy.double()
    rx, rw, _, _ = R.qk_backward(D64, xv, rstd.double(), w.double(), c, s, rot, inter)
    turned = R.rotate(D64.abs(), c.abs(), -s.abs(), rot, inter).abs() + R.rotate(D64.abs(), c.abs(), s.abs(), rot, inter).abs()
    _, _, sx, sw = R.rmsnorm_backward(turned, xv, rstd.double(), w.double())
    near(dx, rx, bf16_bound(rx) + 2.0 ** -18 * sx, "dx")
    near(dw, rw, bf16_bound(rw) + (M * H + 64) * E * sw, "dweight")


def test_an_infinite_element_of_h():
    """x + residual may leave bf16: h is infinite there, and the other elements of y are zeros, as x / inf is."""
    M, N, G = 3, 512, 16
    x = torch.ones(M, N, device="cuda").to(BF)
    x[1, 7] = 3e38
    y, h, q = empty(M, N), empty(M, N), empty(M, N, dtype=U8)
    S, rstd = empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, norm_w(N, 1), EPS, G, y, q, S, rstd, residual=x.clone(), h=h)
    assert torch.isinf(h[1, 7]) and rstd[1] == 0 and torch.isnan(y[1, 7])
    assert not torch.cat((y[1, :7], y[1, 8:])).float().any() and torch.isfinite(y[[0, 2]]).all()
