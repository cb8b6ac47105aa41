"""Few tokens that are all but certain, whose loss and gradient are small differences with a large logit.

Errors that round to nearest do not line up: with E = 2^-24, an exact logit z of positive terms, added pair by pair, has additions
of |z|, twice |z| / 2 and so on, each off by E / sqrt(3) of its sum in the mean square, together by E |z| sqrt(2 / 3), and lse, rounded
once more, by E |z|.  Over n tokens the mean is so off by E |z| / sqrt(n), here allowed six times.  What truncates is off by the same
2^-23 of its size and more in every token."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, E, F32, gen, near, randn, unwritten, workspace
from test_gpu_lm_lce import _built, backward, forward, linear_cross_entropy, linear_cross_entropy_backward  # noqa: F401

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


def certain(M, C, seed, behind=8.5, z=64.0):
    """Every token has a target of logit about z and a rival about `behind` of that; all other logits are small."""
    V = 2 * M + 300
    w = 2 * C ** -0.5 * randn(V, C, seed=seed)
    w[1:2 * M:2] = w[0:2 * M:2] * (1 - behind / z)
    w = w.to(BF)
    t = 2 * torch.arange(M, device="cuda")
    x = (z / 4 * w[t].float()).to(BF)
    order = torch.randperm(V, generator=gen(seed + 1), device="cuda")
    place = torch.empty_like(order)
    place[order] = torch.arange(V, device="cuda")
    return x, w[order].contiguous(), place[t]


@pytest.mark.parametrize("M,C", [(128, 2048), (128, 4096), (100, 1040), (60, 528)])
def test_the_errors_of_a_few_tokens_log_sums_do_not_line_up(M, C):
    x, w, t = certain(M, C, C)
    loss, lse = forward(x, w, t)
    rloss, rlse, z, _ = linear_cross_entropy(x, w, t)
    top = z.amax(1).mean()
    assert (lse - rlse).mean().abs() <= 6 * E * top / M ** 0.5
    # the loss is a sum of terms e^(z - top) of their own: its logits are those of the tensor cores, 128 products in a go
    size = (x.double().abs() @ w.double().abs().T).amax(1)
    near(loss, rloss, rloss * ((136 * 2.0 ** -22 + (C / 128 + 20) * E) * size + (w.shape[0] / 32 + 64 + 2 * 80) * 4 * E), "loss")
    # and lse does not depend on what the targets are
    assert torch.equal(forward(x, w, torch.full_like(t, -1))[1], lse) and torch.equal(forward(x, w, t.flip(0))[1], lse)


@pytest.mark.parametrize("M,C", [(128, 2048), (128, 4096), (100, 1040)])
@pytest.mark.parametrize("own", [False, True])
def test_the_gradient_of_tokens_that_are_all_but_certain(M, C, own):
    """dx = -(1 - p) g (w[t] - w[rival]) but for the others' shares: how far along that.  A target's logit is off by E z sqrt(2 / 3) in
    the mean square (and where lse is the forward pass', both are, and lse rounded: 2 E z at most), over its 1 - p; dz and dx are
    rounded to bf16, 2^-8 / sqrt(3) each; the mean of M tokens by six times the root of their squares' mean over M.  All this is of
    dz w[t], while w[rival] is w[t] (1 - 8.5 / 64), so that dx = -(1 - p) g w[t] 8.5 / 64: of dx it is 64 / 8.5 times as much.

    1 - p is about e^-8.5 = 2e-4; the rival's distance goes with |w[t]|^2, which is off by sqrt(2 / C) of itself in the mean
    square, 13 % at three times that and C = 1040: 1 - p from 6.7e-5 to 6.2e-4."""
    x, w, t = certain(M, C, C + 1)
    rlse, z = linear_cross_entropy(x, w, t)[1:3]
    lse = forward(x, w, t)[1] if own else rlse.float()
    g = torch.rand(M, generator=gen(3), device="cuda") + 0.5
    dx = backward(x, w, t, lse, g)[0].double()
    ref = linear_cross_entropy_backward(x, w, t, rlse if own else lse, g)[0]
    along = (dx * ref).sum(1) / ref.square().sum(1) - 1
    rest = 1 - (z.gather(1, t[:, None]).squeeze(1) - rlse).exp()
    assert rest.min() > 5e-5 and rest.max() < 1e-3
    each = ((2 * E * z.amax(1) / rest).square().mean() + 2 * 2.0 ** -16 / 3).sqrt()
    assert along.mean().abs() <= 64 / 8.5 * 6 * each / M ** 0.5


@pytest.mark.parametrize("M", [1, 2, 5, 128])
def test_the_largest_logit_wherever_it_is(M):
    """Of every token another row of the weight, in any tile, warp and lane: lse is its exact logit and the others' share."""
    V, C = 30011, 272
    w = (0.1 * randn(V, C, seed=1)).to(BF)
    x = randn(M, C, seed=2).to(BF)
    for seed in range(8):
        at = torch.randint(0, V, (M,), generator=gen(seed), device="cuda")
        y = (x.float() + 400 * w[at].float()).to(BF)
        loss, lse = forward(y, w, at)
        rloss, rlse, z, size = linear_cross_entropy(y, w, at)
        near(lse, rlse, (C / 512 + 12) * E * size + 4 * E * rlse, "lse")
        near(loss, rloss, rloss * ((136 * 2.0 ** -22 + (C / 128 + 20) * E) * size + (V / 32 + 64 + 2 * 2000) * 4 * E) + 2.0 ** -126, "loss")
