"""Cross entropy of a linear layer and its gradients on the GPU, through the binding, against float64.

Bounds (U = 2^-8, half a bf16 step relatively; E = 2^-24; the tensor cores add products of bf16 values, exact in float32,
and truncate at worst: 2^-22 per addition):
  * a logit of C terms: D = (C + 8) 2^-22 sum|terms|;
  * lse: D at the row's largest sum of sizes; a sum of V positive terms in chunks, rescaled by factors e^(a - b), each with
    the argument's rounding (2 E |a - b|, |a - b| <= R, the range of the row's logits) and the exponential's 4 E: relatively
    (V / 32 + 64 + 2 R) 4 E, and so absolutely in the logarithm; lse and loss themselves round: 4 E (|top| + |lse|);
  * dz = e^(z - lse) p - [v = t] g: relatively D + (8 + 4 (|z| + |lse|)) E of its first term, 2 E of the second, rounded
    to bf16: U |dz|; dx and dw add V or M terms: (n + 32) 2^-22 sum |dz w|, and round to bf16 once."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, E, F32, U, U8, bf16_bound, gen, linear_cross_entropy, linear_cross_entropy_backward, near, randn, unwritten, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    coat.lib()
    yield
    assert coat.coat_kernel_wait_timeouts(reset=True) == 0


def inputs(M, V, C, seed, index=torch.int64, ld=None, gain=2.0):
    w = (gain * C ** -0.5 * randn(V, C, seed=seed)).to(BF)
    t = torch.randint(0, V, (M,), generator=gen(seed + 1), device="cuda")
    sure = torch.rand(M, 1, generator=gen(seed + 2), device="cuda").square() * 0.3
    x = torch.zeros(M, ld or C, dtype=BF, device="cuda")[:, :C]
    x.copy_(randn(M, C, seed=seed + 3) + sure * C ** 0.5 * w[t].float())
    t[torch.rand(M, generator=gen(seed + 4), device="cuda") < 0.1] = -100
    return x, w, t.to(index)


def forward(x, w, t, ws=None, stream=None):
    M, V = x.shape[0], w.shape[0]
    loss, lse = unwritten(M, dtype=F32), unwritten(M, dtype=F32)
    ws = workspace(coat.coat_linear_cross_entropy_workspace_bytes(M, V)) if ws is None else ws
    coat.coat_linear_cross_entropy(x, w, t, loss, lse, ws, stream=stream)
    return loss, lse


def check_forward(x, w, t):
    loss, lse = forward(x, w, t)
    V, C = w.shape
    rloss, rlse, z, size = linear_cross_entropy(x, w, t)
    R = z.amax(1) - z.amin(1)
    err = (C + 8) * 2.0 ** -22 * size + (V / 32 + 64 + 2 * R) * 4 * E + 4 * E * (z.amax(1).abs() + rlse.abs() + rloss.abs())
    near(lse, rlse, err, "lse")
    near(loss, rloss, torch.where(t < 0, 0.0, 2 * err), "loss")
    return lse


def backward(x, w, t, lse, dloss, dlse=None, piece=0, ws=None, stream=None):
    (M, C), V = x.shape, w.shape[0]
    dx, dw = unwritten(M, C), unwritten(V, C)
    ws = workspace(coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, piece)) if ws is None else ws
    coat.coat_linear_cross_entropy_backward(x, w, t, lse, dloss, dx, dw, ws, dlse=dlse, piece=piece, stream=stream)
    return dx, dw


def check_backward(x, w, t, lse, dloss, dlse=None, piece=0):
    (M, C), V = x.shape, w.shape[0]
    dx, dw = backward(x, w, t, lse, dloss, dlse, piece)
    rx, rw, sx, sw, p, size, z = linear_cross_entropy_backward(x, w, t, lse, dloss, dlse)
    perr = p.abs() * ((C + 8) * 2.0 ** -22 * size + (8 + 4 * (z.abs() + lse.double().abs()[:, None])) * E) * (1 + U) + 2.0 ** -126
    wa, xa = w.double().abs(), x.double().abs()
    g = torch.where(t >= 0, dloss.double().abs(), 0.0)
    ex, ew = perr @ wa, perr.T @ xa
    at = t.long().clamp_min(0)
    ex += 4 * E * g[:, None] * wa[at]
    ew.index_add_(0, at, 4 * E * g[:, None] * xa)
    near(dx, rx, bf16_bound(rx) + (U + (V + 32) * 2.0 ** -22) * (sx + ex) * (1 + U) + ex * (1 + U), "dx")
    near(dw, rw, bf16_bound(rw) + (U + (M + 32) * 2.0 ** -22) * (sw + ew) * (1 + U) + ew * (1 + U), "dw")
    return dx, dw


SIZES = [(97, 700, 64), (128, 129, 1024), (129, 640, 96), (1, 1, 16), (1, 5000, 64), (2, 33, 48), (17, 257, 2048), (33, 1000, 528), (130, 128, 80), (255, 129, 256), (256, 256, 64),
         (257, 513, 144), (300, 4099, 1024), (513, 777, 5120), (1000, 20001, 128), (2048, 512, 1024), (64, 130001, 32)]


@pytest.mark.parametrize("M,V,C", SIZES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_forward(M, V, C, index):
    check_forward(*inputs(M, V, C, M + V, index, ld=C + 24 if index == torch.int32 else None))


@pytest.mark.parametrize("M,V,C", SIZES)
@pytest.mark.parametrize("zloss,piece", [(False, 0), (True, 256), (True, 1000)])
def test_backward(M, V, C, zloss, piece):
    if piece == 256 and V > 30000:
        piece = 4096
    x, w, t = inputs(M, V, C, M * V, torch.int32 if zloss else torch.int64, ld=C + 8 if zloss else None)
    lse = linear_cross_entropy(x, w, t)[1].float()
    dloss = randn(M, seed=5).abs() / M
    check_backward(x, w, t, lse, dloss, 1e-3 * randn(M, seed=6) if zloss else None, piece)


@pytest.mark.parametrize("M,V,C", [(700, 1300, 272), (100, 1300, 272), (20, 30000, 64), (5000, 100, 64), (257, 513, 1040)])
def test_every_operand_in_whole_numbers(M, V, C):
    """dz of 0, +-1 by choice of lse and gradients, whole numbers elsewhere: sums are exact in every order, so an element
    that is missed, doubled or misplaced in any tile, piece or part shows.

    x = 0: every logit is 0; lse = 0: e^0 = 1 for every column; dloss = 1: dz = 1 - [v = t]."""
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    w = torch.randint(-1, 2, (V, C), generator=gen(1), device="cuda").to(BF)
    t = torch.randint(0, V, (M,), generator=gen(2), device="cuda")
    dloss, lse = torch.ones(M, device="cuda"), torch.zeros(M, device="cuda")
    want = (w.double().sum(0) - w.double()[t]).to(BF)
    for piece in (0, 256, 512, 1280):
        dx, dw = backward(x, w, t, lse, dloss, piece=piece)
        assert torch.equal(dx, want) and not dw.any()
    # and W = 0 with x of whole numbers: dw[v] = sum over tokens of x - those with the target v
    w = torch.zeros(V, C, dtype=BF, device="cuda")
    x = torch.randint(-1, 2, (M, C), generator=gen(3), device="cuda").to(BF)
    want = x.double().sum(0).repeat(V, 1).index_add(0, t, -x.double()).to(BF)
    for piece in (0, 256, 768):
        dx, dw = backward(x, w, t, lse, dloss, piece=piece)
        assert torch.equal(dw, want) and not dx.any()


@pytest.mark.parametrize("M", [100, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_what_a_padded_token_holds_does_not_count(M, bad):
    """Rows without a target and without gradients, whose logits are NaN or infinite: loss 0, zeros in dx, and every other row
    as it is without them."""
    V, C = 400, 64
    x, w, t = inputs(M, V, C, 1)
    rest = t >= 0
    loss, lse = forward(x, w, t)
    padded = x.clone()
    padded[~rest] = bad
    loss2, lse2 = forward(padded, w, t)
    assert not loss2[~rest].any() and torch.equal(loss2, loss) and torch.equal(lse2[rest], lse[rest])
    dloss = torch.full((M,), 1 / M, device="cuda")
    dx, _ = backward(x, w, t, lse, dloss)
    dx2, _ = backward(padded, w, t, lse2, dloss)
    assert torch.equal(dx2, dx) and not dx2[~rest].any()
    weights = torch.where(torch.arange(M, device="cuda") % 3 == 0, 0.0, dloss)      # tokens with a target and no weight
    dx3, _ = backward(x, w, t, lse, weights)
    assert not dx3[::3].any()


def test_logits_of_one_hot_rows_are_the_weights():
    """x = unit vectors: a row's logits are a column of W, so lse and loss name it; W is different everywhere."""
    V, C = 1000, 144
    x = torch.eye(C, dtype=BF, device="cuda")
    w = (4 * randn(V, C, seed=1)).to(BF)
    t = torch.randint(0, V, (C,), generator=gen(2), device="cuda")
    loss, lse = forward(x, w, t)
    ref = torch.logsumexp(w.double(), 0)
    assert ((lse - ref).abs() <= 2.0 ** -18 * ref.abs().clamp_min(1)).all()
    assert ((loss - (ref - w.double()[t, torch.arange(C, device="cuda")])).abs() <= 2.0 ** -17 * ref.abs().clamp_min(8)).all()


def test_tokens_without_a_target():
    M, V, C = 100, 300, 64
    x, w, t = inputs(M, V, C, 1)
    none = torch.full_like(t, -1)
    loss, lse = forward(x, w, none)
    assert not loss.any() and torch.equal(lse, forward(x, w, t)[1])
    dloss = torch.full((M,), float("nan"), device="cuda")          # does not count
    dx, dw = backward(x, w, none, lse, dloss)
    assert not dx.any() and not dw.any()
    mixed = t.clone()
    mixed[::2] = -(1 << 40)
    dloss = torch.where(mixed < 0, float("nan"), 0.25)
    check_backward(x, w, mixed, lse, dloss)
    check_backward(x, w, mixed, lse, dloss, dlse=randn(M, seed=1))
    assert not backward(x, w, mixed, lse, dloss)[0][::2].any()


def test_targets_past_the_vocabulary_give_nan():
    M, V, C = 40, 200, 64
    x, w, t = inputs(M, V, C, 1)
    t[7], t[21] = V, 1 << 40
    loss, lse = forward(x, w, t)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[7, 21]] = True
    assert torch.equal(loss.isnan(), bad) and lse.isfinite().all()
    dx, dw = backward(x, w, t, lse, torch.ones(M, device="cuda"))
    assert torch.equal(dx.isnan().any(1), bad) and dw.isnan().any()


def test_certain_tokens():
    """A target's logit far above all others: the loss is small and exact to its own size, and nothing overflows."""
    M, V, C = 64, 3000, 64
    w = randn(V, C, seed=1).to(BF)
    t = torch.randint(0, V, (M,), generator=gen(2), device="cuda")
    x = (torch.linspace(0.02, 200, M, device="cuda")[:, None] * w[t].float()).to(BF)
    lse = check_forward(x, w, t)
    loss = forward(x, w, t)[0]
    assert (loss >= 0).all() and (loss[40:] < 1e-6).all()
    check_backward(x, w, t, lse, torch.ones(M, device="cuda"))


def test_logits_of_minus_infinity_and_of_the_types_lowest_value():
    """Columns that a huge negative weight masks, whole tiles of them first: they have no share."""
    M, V, C = 70, 1500, 32
    x, w, t = inputs(M, V, C, 3)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    free = torch.randperm(V - 700, generator=gen(4), device="cuda")[:100] + 700
    t = free[torch.randint(0, 100, (M,), generator=gen(5), device="cuda")]
    lowest = torch.finfo(BF).min
    ref = None
    for low in (-1e4, lowest, -float("inf")):
        masked = w.clone()
        masked[:, 0] = low
        masked[free, 0] = 0.0
        if low == -float("inf"):       # -inf times 1, and 0 elsewhere: the products are no NaN
            masked[masked[:, 0] == low, 1:] = 0.0
        loss, lse = forward(x, masked, t)
        ref = lse if ref is None else ref
        assert torch.equal(lse, ref) and loss.isfinite().all()
        if low != -float("inf"):
            dx, dw = backward(x, masked, t, lse, torch.ones(M, device="cuda"))
            assert dx.isfinite().all() and dw.isfinite().all()
            out = torch.ones(V, dtype=torch.bool, device="cuda")
            out[free] = False
            assert not dw[out].any()


def test_the_same_bits_every_time_and_whatever_the_workspace_holds():
    M, V, C = 700, 2100, 256
    x, w, t = inputs(M, V, C, 1)
    loss, lse = forward(x, w, t)
    dloss = torch.full((M,), 1 / M, device="cuda")
    dx, dw = backward(x, w, t, lse, dloss, piece=512)
    for fill in (0, 0x7F, 0xC0):
        ws = torch.full((coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, 512),), fill, dtype=U8, device="cuda")
        a, b = forward(x, w, t, ws=ws)
        assert torch.equal(a, loss) and torch.equal(b, lse)
        a, b = backward(x, w, t, lse, dloss, piece=512, ws=ws)
        assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("shift", [8, 16])
def test_pointers_of_16_bytes(shift):
    M, V, C = 140, 600, 80
    x, w, t = inputs(M, V, C, 2)

    def view(v, dtype=BF, k=1):
        s = torch.empty(v.numel() + shift * k, dtype=dtype, device="cuda")[shift * k:].view(v.shape)
        return s.copy_(v)
    loss, lse = forward(x, w, t)
    dloss = torch.full((M,), 1 / M, device="cuda")
    dx, dw = backward(x, w, t, lse, dloss, piece=256)
    n = coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, 256)
    ws = torch.empty(n + 2 * shift, dtype=U8, device="cuda")[2 * shift:]
    x2, w2 = view(x), view(w)
    dx2, dw2 = view(dx.clone().fill_(7)), view(dw.clone().fill_(7))
    coat.coat_linear_cross_entropy_backward(x2, w2, t, lse, dloss, dx2, dw2, ws, piece=256)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_weight_past_2_31_elements():
    M, V, C = 3, 140000, 16384
    w = torch.zeros(V, C, dtype=BF, device="cuda")
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    x[:, 0] = torch.tensor([1.0, 2.0, 4.0])
    w[V - 1, 0], w[131075, 0], w[5, 0] = 8.0, 4.0, 2.0
    t = torch.tensor([V - 1, 131075, 5], device="cuda")
    loss, lse = forward(x, w, t)
    k = x[:, 0].double()[:, None] * torch.tensor([8.0, 4.0, 2.0], device="cuda", dtype=torch.float64)
    ref = (k.exp().sum(1) + V - 3).log()
    assert ((lse - ref).abs() < 1e-5).all() and ((loss - (ref - k.diagonal())).abs() < 1e-5).all()
    dx, dw = unwritten(M, C), unwritten(V, C)
    ws = workspace(coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C))
    coat.coat_linear_cross_entropy_backward(x, w, t, lse, torch.ones(M, device="cuda"), dx, dw, ws)
    p = (k - ref[:, None]).exp()
    p -= torch.eye(3, device="cuda", dtype=torch.float64)
    want = (p * x[:, 0].double()[:, None]).sum(0)
    assert ((dw[[V - 1, 131075, 5], 0].double() - want).abs() <= 2.0 ** -6 * (p.abs() * x[:, 0].double()[:, None]).sum(0)).all()
    others = (x[:, 0].double() * (-ref).exp()).sum().item()
    assert ((dw[[0, 131071, 131076, V - 2], 0].double() - others).abs() <= 2.0 ** -6 * others).all() and not dw[:, 1:].any()
    assert ((dx[:, 0].double() - (p * torch.tensor([8.0, 4.0, 2.0], device="cuda", dtype=torch.float64)).sum(1)).abs() <= 0.1).all()


def test_captured_and_replayed_on_another_stream():
    M, V, C = 300, 900, 96
    x, w, t = inputs(M, V, C, 1)
    loss, lse = unwritten(M, dtype=F32), unwritten(M, dtype=F32)
    dx, dw, dloss = unwritten(M, C), unwritten(V, C), torch.full((M,), 1 / M, device="cuda")
    ws = workspace(max(coat.coat_linear_cross_entropy_workspace_bytes(M, V),
                       coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, 512)))

    def both():
        coat.coat_linear_cross_entropy(x, w, t, loss, lse, ws)
        coat.coat_linear_cross_entropy_backward(x, w, t, lse, dloss, dx, dw, ws, piece=512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (7, 8):
        for a, b in zip((x, w, t), inputs(M, V, C, seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        rl, rs = forward(x, w, t)
        rx, rw = backward(x, w, t, rs, dloss, piece=512)
        assert torch.equal(loss, rl) and torch.equal(lse, rs) and torch.equal(dx, rx) and torch.equal(dw, rw)


def test_gradient_is_that_of_differences():
    """(L(x + d) - L(x - d)) / 2 = <dx, d> + O(d^3) for L = sum g loss + h lse in float64 of the library's own inputs."""
    M, V, C = 40, 500, 64
    x, w, t = inputs(M, V, C, 9)
    g, h = randn(M, seed=1).abs(), 0.1 * randn(M, seed=2)
    lse = linear_cross_entropy(x, w, t)[1].float()
    dx, dw = backward(x, w, t, lse, g, h)

    def L(x, w):
        loss, lse, _, _ = linear_cross_entropy(x, w, t)
        return (g.double() * loss + h.double() * lse).sum()
    for which, grad, base in ((0, dx, x), (1, dw, w)):
        d = 1e-4 * torch.randn(base.shape, generator=gen(which + 3), device="cuda", dtype=torch.float64)
        args = [[x.double(), w.double()], [x.double(), w.double()]]
        args[0][which] = args[0][which] + d
        args[1][which] = args[1][which] - d
        got, want = (grad.double() * d).sum(), (L(*args[0]) - L(*args[1])) / 2
        # dz and the gradient are rounded to bf16: errors of U of every term, whose signs are those of d, at random
        sizes = linear_cross_entropy_backward(x, w, t, lse, g, h)[2 + which]
        assert (got - want).abs() <= 12 * U * ((sizes * d).square().sum().sqrt()) + 1e-9


def test_refusals():
    x, w, t = inputs(20, 50, 32, 1)
    loss, lse, ws = unwritten(20, dtype=F32), unwritten(20, dtype=F32), workspace(1 << 16)
    with pytest.raises(TypeError, match="dtype"):
        coat.coat_linear_cross_entropy(x.float(), w, t, loss, lse, ws)
    with pytest.raises(TypeError, match="dtype"):
        coat.coat_linear_cross_entropy(x, w, t.float(), loss, lse, ws)
    with pytest.raises(ValueError, match="weight must have"):
        coat.coat_linear_cross_entropy(x, w[:, :16].contiguous(), t, loss, lse, ws)
    with pytest.raises(ValueError, match="together"):
        coat.coat_linear_cross_entropy(x.T.contiguous().T, w, t, loss, lse, ws)
    with pytest.raises(ValueError, match="targets"):
        coat.coat_linear_cross_entropy(x, w, t[:5], loss, lse, ws)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_linear_cross_entropy(x, w, t, loss, lse, ws[:16])
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_linear_cross_entropy(x, w, t, loss, loss, ws)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_linear_cross_entropy_backward(x, w, t, lse, loss, x, unwritten(50, 32), ws)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_linear_cross_entropy_backward(x, w, t, lse, loss, unwritten(20, 32), unwritten(50, 32), ws, piece=-1)


@pytest.mark.parametrize("M,V,C", [(100, 3000, 256), (700, 3000, 256)])
@pytest.mark.parametrize("first", [0, 40])
def test_a_mean_over_the_tokens_is_not_off_by_the_rounding_of_its_factor(M, V, C, first):
    """The targets' dz are all but -g: with one g for all tokens, halfway between two bf16 values, its rounding (2^-8 of it)
    would be that of dx and dw.  Errors that do not line up are, for values spread over a binade, 2^-8 sqrt(0.541 / 3) = 0.00166
    of themselves in the mean square at each rounding; dz and the output are two: 0.00235, and a tenth for the spread."""
    x, w, t = inputs(M, V, C, 21, gain=1.0)
    t = torch.randint(0, V, (M,), generator=gen(5), device="cuda")
    t[:first] = -1                                         # the first tokens have no target
    g = torch.full((M,), (1 + 2.0 ** -8 + 2.0 ** -20) * 2.0 ** -13, device="cuda")
    lse = linear_cross_entropy(x, w, t)[1].float()
    for piece in (0, 512):
        dx, dw = check_backward(x, w, t, lse, g, piece=piece)
        rx, rw = linear_cross_entropy_backward(x, w, t, lse, g)[:2]
        for got, ref in ((dx, rx), (dw, rw)):
            assert (got.double() - ref).norm() / ref.norm() <= 0.0026


def test_gradients_that_are_no_numbers_to_divide_by():
    """Gradients below any scale, zeros, and one that is infinite or NaN: each stays what it is, in its own row."""
    M, V, C = 70, 300, 64
    x, w, t = inputs(M, V, C, 22)
    t = t.clamp_min(0)
    lse = linear_cross_entropy(x, w, t)[1].float()
    zero = torch.zeros(M, device="cuda")
    assert not any(d.any() for d in backward(x, w, t, lse, zero))
    tiny = torch.full((M,), 2.0 ** -120, device="cuda")
    dx, dw = backward(x, w, t, lse, tiny)
    assert dx.isfinite().all() and dw.isfinite().all()
    check_backward(x, w, t, lse, torch.where(torch.arange(M, device="cuda") < 5, 0.0, 0.3).float())
    for bad in (float("inf"), float("nan")):
        g = torch.full((M,), 0.3, device="cuda")
        g[0] = bad
        dx, _ = backward(x, w, t, lse, g)
        g[0] = 0.0
        ref, _ = backward(x, w, t, lse, g)
        assert not dx[0].isfinite().all() and torch.equal(dx[1:], ref[1:])


@pytest.mark.parametrize("M,V,at", [(3, 40001, 7), (129, 40001, 40000), (200, 97, 40), (1, 2, 1)])
@pytest.mark.parametrize("ahead", [10.0, 15.0, 20.0])
def test_loss_of_a_certain_token_is_that_of_the_others_terms(M, V, at, ahead):
    """The target's logit is `ahead` of all others, exactly: loss = log(1 + (V - 1) e^-ahead), of terms as small as 2e-9.  At most
    31 of them share 32 columns with the target's 1, and may be lost beside it; of 16 additions to the 1, and of 32 columns'
    sum less 1, each may be off by 2^-23, but by no more than what is added.  The others: joins of V / 32 sums, the exponential's
    error and its argument's, 2 ahead."""
    C = 64
    w = torch.zeros(V, C, dtype=BF, device="cuda")
    w[at, 3] = ahead / 2
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    x[:, 3] = 2
    loss, lse = forward(x, w, torch.full((M,), at, device="cuda"))
    term = torch.exp(torch.tensor(-ahead, dtype=torch.float64)).item()
    ref = torch.log1p(torch.tensor((V - 1) * term, dtype=torch.float64)).expand(M).cuda()
    err = 31 * min(term, 2.0 ** -23) + ref * (V / 32 + 64 + 2 * ahead) * 4 * E
    near(loss, ref, err, "loss")
    near(lse, ref + ahead, err + 4 * E * ahead, "lse")


@pytest.mark.parametrize("M", [100, 300])
def test_logits_that_are_not_numbers_give_nan_in_their_rows_alone(M):
    x, w, t = inputs(M, 700, 128, 23)
    t = t.clamp_min(0)
    good = forward(x, w, t)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[[0, M - 1], 5] = bad
        loss, lse = forward(y, w, t)
        assert loss[[0, M - 1]].isnan().all() and lse[[0, M - 1]].isnan().all()
        assert torch.equal(loss[1:-1], good[0][1:-1]) and torch.equal(lse[1:-1], good[1][1:-1])


@pytest.mark.parametrize("M,V", [(1, 20001), (33, 25001), (128, 30001), (40, 47003), (100, 38913), (65, 19457)])
def test_few_tokens_in_tiles_of_fewer_rows_of_the_weight(M, V):
    """More tiles of the weight's rows than pairs of multiprocessors: every row counts once, wherever a tile ends."""
    check_forward(*inputs(M, V, 48, V, torch.int32))
    test_every_operand_in_whole_numbers(M, V, 32)
    x, w, t = inputs(M, V, 32, V)
    x[:] = 0
    x[:, 7] = 1
    w[:, 7] = torch.arange(V, device="cuda").remainder(5).to(BF)     # the logits, exactly, of which the sum is known
    loss, lse = forward(x, w, t)
    count = torch.bincount(torch.arange(V, device="cuda").remainder(5), minlength=5).double()
    want = (count * torch.exp(torch.arange(5, device="cuda").double())).sum().log().expand(M)
    near(lse, want, torch.full_like(want, (V / 32 + 64 + 8) * 4 * E + 4 * E * 20), "lse")
    near(loss, torch.where(t < 0, 0.0, want - w[t.clamp_min(0), 7].double()),
         torch.where(t < 0, 0.0, (V / 32 + 64 + 8) * 4 * E + 4 * E * 24).double(), "loss")


@pytest.mark.parametrize("V", [19456, 19451])
def test_tiles_with_all_their_columns(V):
    """Two waves of tiles of 256 x 256, the last one of 251 columns: targets in every place of a tile, and rows whose logits are all
    or in part -inf, not numbers, or far ahead of each other."""
    M, C = 512, 64
    x, w, t = inputs(M, V, C, 31)
    t = (torch.arange(M, device="cuda") * 38 + 11) % V          # every column of a tile is someone's target
    t[::2] = torch.arange(M // 2, device="cuda") + V - 256
    check_forward(x, w, t)
    good = forward(x, w, t)
    w[:, 60:] = 0
    w[:, 60] = -3e38
    w[1::2, 61] = -3e38
    w[::3, 62] = 10.0
    y = x.clone()
    y[:, 60:] = 0
    plain = forward(y, w, t)
    for r, c, v in ((3, 60, 3e38), (4, 61, 3e38), (5, 62, 2.0), (6, 0, float("nan")), (7, 1, float("inf"))):
        y[r, c] = v
    loss, lse = forward(y, w, t)
    assert lse[3] == -float("inf") and not loss[3].isfinite()
    z = y.double() @ w.double().T
    size = y.abs().double() @ w.abs().double().T
    for r, keep in ((4, torch.arange(V, device="cuda") % 2 == 0), (5, torch.ones(V, dtype=torch.bool, device="cuda"))):
        ref = torch.logsumexp(z[r][keep], 0)
        err = (C + 8) * 2.0 ** -22 * size[r][keep].amax() + (V / 32 + 64 + 100) * 4 * E + 4 * E * ref.abs()
        assert (lse[r].double() - ref).abs() <= err
    assert loss[[6, 7]].isnan().all() and lse[[6, 7]].isnan().all()
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[3:8] = False
    assert torch.equal(loss[rest], plain[0][rest]) and torch.equal(lse[rest], plain[1][rest])
    assert good[0].isfinite().all() and good[1].isfinite().all()


@pytest.mark.parametrize("first", [1023, 1024, 1500, 2990])
def test_a_mean_over_the_tokens_behind_many_without_a_target(first):
    """A long prompt without targets: the factor is that of the first token that has one, wherever it stands.  The bound is that of
    test_a_mean_over_the_tokens_is_not_off_by_the_rounding_of_its_factor; with the factor's own rounding, 2^-8, errors of all
    target's terms line up, and dx and dweight are 0.0033 and more off."""
    M, V, C = 3000, 3000, 256
    x, w, _ = inputs(M, V, C, 21, gain=1.0)
    t = torch.randint(0, V, (M,), generator=gen(5), device="cuda")
    t[:first] = -100
    g = torch.full((M,), (1 + 2.0 ** -8 + 2.0 ** -20) * 2.0 ** -13, device="cuda")
    g[:first:2] = float("nan")                                # of a token without a target it does not count
    lse = linear_cross_entropy(x, w, t)[1].float()
    for piece in (0, 512):
        dx, dw = check_backward(x, w, t, lse, g, piece=piece)
        rx, rw = linear_cross_entropy_backward(x, w, t, lse, g)[:2]
        for got, ref in ((dx, rx), (dw, rw)):
            assert (got.double() - ref).norm() / ref.norm() <= 0.0026
