"""Few tokens that are all but certain, whose loss and gradient are small differences with a large logit."""
import pytest
import torch

from _lm_ref import BF, E, near
from test_gpu_lm_lce import _built, forward  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,V,at", [(1, 97, 40), (1, 32, 0), (3, 97, 96), (40, 20011, 20010), (128, 97, 5)])
@pytest.mark.parametrize("ahead", [10.0, 15.0, 20.0])
def test_no_term_is_summed_with_the_largest_ones(M, V, at, ahead):
    """The target's logit is `ahead` of all others, exactly: loss = log(1 + (V - 1) e^-ahead), the terms that share 32 rows with it
    among them.  V / 32 sums and their joins, the exponential's error and its argument's, 2 ahead."""
    C = 64
    w = torch.zeros(V, C, dtype=BF, device="cuda")
    w[at, 3] = ahead / 2
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    x[:, 3] = 2
    loss, lse = forward(x, w, torch.full((M,), at, device="cuda"))
    ref = torch.log1p((V - 1) * torch.exp(torch.tensor(-ahead, dtype=torch.float64))).expand(M).cuda()
    err = ref * (V / 32 + 64 + 2 * ahead) * 4 * E
    near(loss, ref, err, "loss")
    near(lse, ref + ahead, err + 4 * E * ahead, "lse")
