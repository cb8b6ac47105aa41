"""The cross entropy's gradients at sizes that take several pieces of the vocabulary by themselves, and past 2^31 elements.

In whole numbers: x = 0, lse = 0 and dloss = 1 make dz = 1 - [v = t], so that dx = sum of W - W[t], exact in every order; W = 0 makes
dweight[v] = sum of x - those with the target v."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, gen, unwritten
from test_gpu_lm_lce import _built, backward, check_backward, inputs, linear_cross_entropy  # noqa: F401  (_built: module fixture)

pytestmark = pytest.mark.gpu


def whole(*shape, seed):
    return torch.randint(-1, 2, shape, generator=gen(seed), device="cuda", dtype=torch.int8).to(BF)


def check_whole_numbers(M, V, C, piece=0):
    t = torch.randint(0, V, (M,), generator=gen(2), device="cuda")
    dloss, lse = torch.ones(M, device="cuda"), torch.zeros(M, device="cuda")
    zero = torch.zeros(M, C, dtype=BF, device="cuda")
    w = whole(V, C, seed=1)
    dx, dw = backward(zero, w, t, lse, dloss, piece=piece)
    total = w.float().sum(0)                              # whole numbers below 2^24: exact
    for m in range(0, M, 8192):
        assert torch.equal(dx[m:m + 8192], (total - w[t[m:m + 8192]].float()).to(BF))
    assert not dw.any()
    del dx, dw, w, zero
    x = whole(M, C, seed=3)
    dx, dw = backward(x, torch.zeros(V, C, dtype=BF, device="cuda"), t, lse, dloss, piece=piece)
    assert not any(dx[m:m + 8192].any() for m in range(0, M, 8192))
    want = torch.zeros(C, device="cuda")
    taken = torch.zeros(V, C, device="cuda")
    for m in range(0, M, 8192):
        part = x[m:m + 8192].float()
        want += part.sum(0)
        taken.index_add_(0, t[m:m + 8192], part)
    assert torch.equal(dw, (want - taken).to(BF))


def test_several_pieces_by_default():
    M, V, C = 16384, 33000, 64
    one = coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, V)
    assert coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C) < one / 2   # three pieces of 11008 rows
    check_whole_numbers(M, V, C)
    x, w, t = inputs(M, V, C, 1)
    lse = linear_cross_entropy(x, w, t)[1].float()
    check_backward(x, w, t, lse, torch.rand(M, generator=gen(4), device="cuda") / M)


def test_a_piece_of_more_than_2_31_elements():
    check_whole_numbers(70001, 32768, 16, piece=32768)


@pytest.mark.parametrize("V", [97, 700])
def test_tokens_of_more_than_2_31_elements(V):
    check_whole_numbers(140001, V, 16384, piece=0 if V == 97 else 256)


def test_the_loss_of_tokens_of_more_than_2_31_elements():
    """Unit rows: a token's logits are a column of W, so rows of x on both sides of 2^31 elements name theirs."""
    M, V, C = 140001, 97, 16384
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    at = torch.arange(M, device="cuda") * 7 % C
    x[torch.arange(M, device="cuda"), at] = 1
    w = (4 * torch.randn(V, C, generator=gen(1), device="cuda")).to(BF)
    t = torch.arange(M, device="cuda") % V
    loss, lse = unwritten(M, dtype=torch.float32), unwritten(M, dtype=torch.float32)
    ws = torch.empty(coat.coat_linear_cross_entropy_workspace_bytes(M, V), dtype=torch.uint8, device="cuda")
    coat.coat_linear_cross_entropy(x, w, t, loss, lse, ws)
    ref = torch.logsumexp(w.double(), 0)
    assert ((lse - ref[at]).abs() <= 2.0 ** -18 * ref[at].abs().clamp_min(1)).all()
    assert ((loss - (ref[at] - w.double()[t, at])).abs() <= 2.0 ** -17 * ref[at].abs().clamp_min(16)).all()
