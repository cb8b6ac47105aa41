"""What the header says of the rounding inside the operators with 8-bit activation checkpoints.

The weight gradient's operand goes to the tensor cores as RN_bf16(E4M3(q) RN(scale row_scale)).  Against the product of
that operand in float64 nothing is left but the float32 sum of M terms, truncating at worst, (M + 8) 2^-22 of sum|dy X|,
and the result's own rounding: at these token counts, less than half of what one token adds where the terms are alike.

The gated unit's sigmoid is read from the product's scale, which is float32: max|g s u| / 448."""
import pytest
import torch

import _ckpt_ref as R
from test_gpu_ckpt import BF, E, E4M3, EPS, F32, U, U8, acts, bf16_bound, checkpoint, empty, grads, near, norm_w
from test_gpu_ckpt import _built  # noqa: F401  (module fixture)
from test_gpu_ckpt_wgrad import weight_grad
import coat_fp8_adamw_gb300 as coat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,G,row,col", [(5, 72, 80, 16, True, False), (64, 264, 272, 8, False, True), (257, 520, 400, 16, True, True),
                                             (640, 1016, 1024, 128, True, True), (1000, 2048, 2048, 32, True, False),
                                             (1111, 2048, 2048, 16, False, False), (1000, 2560, 3840, 64, True, True)])
def test_the_rounded_operand_is_all_that_is_lost(M, N, K, G, row, col):
    x, dy = acts(M, K, M + K), grads(M, N, M + N)
    q, S, _ = checkpoint(x, G)
    r = torch.rsqrt(x.float().square().mean(-1) + EPS) if row else None
    c = norm_w(K, 8) if col else None
    f = S if r is None else S * r[:, None]                        # float32
    X = (q.view(E4M3).float() * f.repeat_interleave(G, 1)).to(BF).double()
    ref, size = R.weight_grad(dy.double(), X, None, None if c is None else c.double())
    near(weight_grad(dy, q, S, G, r, c), ref, bf16_bound(ref) + (M + 8) * 2.0 ** -22 * size, "dw")
    # and with it, the bound that the header gives
    ref, size = R.weight_grad(dy.double(), R.dequantize(q.view(E4M3).double(), S.double(), G), None if r is None else r.double(),
                              None if c is None else c.double())
    near(weight_grad(dy, q, S, G, r, c), ref, U * ref.abs() + (U + (M + 8) * 2.0 ** -22) * size + 2.0 ** -133, "dw")


def test_the_sigmoid_is_as_near_as_the_header_says():
    """Groups of one value each, +-1.75 2^j, which a checkpoint holds exactly, as it does u = 1.75."""
    G, j = 8, torch.arange(-24, 8, device="cuda", dtype=torch.float64)
    g = torch.cat((1.75 * torch.exp2(j), -1.75 * torch.exp2(j)))
    M, N = g.numel(), 16
    gate = g[:, None].expand(M, N).contiguous().to(BF)
    (gq, gs, gv), (uq, us, uv) = checkpoint(gate, G), checkpoint(torch.full_like(gate, 1.75), G)
    assert torch.equal(gv[:, 0], g) and (uv == 1.75).all()
    hq, hs = empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)
    coat.coat_swiglu_ckpt_backward(torch.ones_like(gate), gq, gs, uq, us, G, empty(M, N), empty(M, N), h_q=hq, h_scale=hs)
    ref = g.abs() * torch.special.expit(g) * 1.75 / 448
    gone = g < -87.3
    assert (hs[gone] == 0).all() and (hs[~gone] > 0).all()
    # two products and the division by 448 beside the sigmoid
    near(hs[~gone], ref[~gone, None].expand(-1, N // G), ((g.abs() + 8) * 2 * E + 4 * E)[~gone, None] * ref[~gone, None], "scale")
