"""The norm's backward pass waits for its own copies with a limit: no wait gives up in ordinary calls, whatever the
number of rows, rounds and stages, and what a call leaves does not differ from the next one's."""
import pytest
import torch

import _ckpt_ref as R
import coat_fp8_adamw_gb300 as coat
from test_gpu_ckpt import EPS, acts, checkpoint, empty, grads, norm_w, workspace
from test_gpu_ckpt import _built  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu


# teams of one warp to one team of 32 warps; one, two and three blocks per SM; rings of two to four stages
@pytest.mark.parametrize("N,G", [(16, 16), (1024, 64), (3200, 128), (4096, 16), (5120, 128), (8192, 32), (12288, 128), (16384, 64)])
@pytest.mark.parametrize("res", [False, True])
def test_no_wait_gives_up(N, G, res):
    coat.coat_kernel_wait_timeouts(reset=True)
    for M in (1, 2, 153, 1500, 4099):
        x, w, dy = acts(M, N, M + N), norm_w(N, 6), grads(M, N, M + 3)
        q, S, _ = checkpoint(x, G)
        rstd = R.rmsnorm(x.double(), w.double(), EPS)[1].float()
        dres = grads(M, N, M + 4) if res else None
        ws = workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N))
        out = []
        for _ in range(2):
            out.append((empty(M, N), empty(N)))
            coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, *out[-1], ws, dresidual=dres)
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
        assert torch.isfinite(out[0][0]).all() and torch.isfinite(out[0][1]).all()
        assert coat.coat_kernel_wait_timeouts() == 0
