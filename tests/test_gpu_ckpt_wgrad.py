"""The weight gradient where a single token, column or part shows.

Whole numbers: dy and the checkpoint hold 0 and +-1, the scales and factors powers of two, so thinly that every sum is
exact in float32 and in bf16; the result has to be the exact one, whatever the order, the tiles and the parts."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from test_gpu_ckpt import BF, E4M3, U8, empty, gen, workspace
from test_gpu_ckpt import _built  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu


def weight_grad(dy, q, S, G, r=None, c=None):
    (M, N), K = dy.shape, q.shape[1]
    dw = empty(N, K)
    ws = workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K))
    coat.coat_ckpt_weight_grad(dy, q, S, G, dw, ws, row_scale=r, col_scale=c)
    torch.cuda.synchronize()
    assert coat.coat_kernel_wait_timeouts() == 0
    return dw


def thin(M, N, seed):
    """0 and +-1, about 24 products of two such columns' entries that are not 0."""
    p = min(1.0, (24 / M) ** 0.5)
    on = torch.rand(M, N, generator=gen(seed), device="cuda") < p
    return on * (1.0 - 2.0 * (torch.rand(M, N, generator=gen(seed + 1), device="cuda") < 0.5))


# one tile, several, tiles that are split along the tokens, more tiles than pairs, ragged edges
@pytest.mark.parametrize("N,K", [(8, 128), (256, 256), (520, 384), (1024, 1024), (2048, 2176), (4096, 1408), (2560, 3840)])
@pytest.mark.parametrize("G", [8, 16, 32, 64, 128])
def test_whole_numbers_are_exact(N, K, G):
    for M in (1, 16, 63, 64, 65, 511, 513, 1111, 2048, 4097):
        dy, x = thin(M, N, M + N), thin(M, K, M + K + 2)
        S = torch.exp2(-torch.randint(0, 2, (M, K // G), generator=gen(M), device="cuda").float())
        r = torch.exp2(torch.randint(0, 2, (M,), generator=gen(M + 1), device="cuda").float())
        c = torch.exp2(torch.randint(-3, 4, (K,), generator=gen(K), device="cuda").float())
        q = x.to(E4M3).view(U8)
        dw = weight_grad(dy.to(BF), q, S, G, r, c)
        X = x.double() * S.double().repeat_interleave(G, 1) * r.double()[:, None]
        ref = (dy.double().T @ X) * c.double()
        assert torch.equal(ref.to(BF).double(), ref)              # the inputs are as thin as they should be
        assert torch.equal(dw.double(), ref), f"M={M}"
