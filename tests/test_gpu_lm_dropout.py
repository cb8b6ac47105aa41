"""Dropout on the GPU, through the binding, against the generator's definition.

The mask is the definition's, element for element.  A kept element is one float32 product (and one addition), rounded to
bf16: U (1 + U) |ref| + 2 E (|x scale| + |residual|), U = 2^-8, E = 2^-24."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, E, bf16_bound, draws, near, randn, threshold, unwritten

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    coat.lib()


def key(a, b):
    return torch.tensor([a, b], dtype=torch.int64, device="cuda")


def want(x, p, rng, start=0, residual=None):
    T = threshold(p)
    keep = (draws(rng.tolist(), start, x.numel()) >= T).view(x.shape).to(x.device)
    y = torch.where(keep, x.double() * (65536 / (65536 - T)), 0.0)
    return (y if residual is None else y + residual.double()), keep, y.abs()


SIZES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 4095, 4096, 4097, 16 * 4096 + 5, (33, 2048), (3, 5, 80), 1000003]


@pytest.mark.parametrize("shape", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_both_directions(shape, p):
    shape = shape if isinstance(shape, tuple) else (shape,)
    x, r, rng = randn(*shape, seed=1).to(BF), randn(*shape, seed=2).to(BF), key(0x123456789ABCDEF, 77)
    for res in (None, r):
        y = unwritten(*shape)
        coat.coat_dropout(x, p, rng, y, residual=res)
        ref, keep, size = want(x, p, rng, residual=res)
        near(y, ref, bf16_bound(ref) + 2 * E * (size + ref.abs()), "y")
        assert torch.equal(y[~keep], torch.zeros_like(y[~keep]) if res is None else res[~keep])
    dx = unwritten(*shape)
    coat.coat_dropout_backward(x, p, rng, dx)
    ref, keep, size = want(x, p, rng)
    near(dx, ref, bf16_bound(ref) + 2 * E * size, "dx")
    assert not dx[~keep].any()
    if p == 0.0:
        assert torch.equal(dx, x) and keep.all()


@pytest.mark.parametrize("a,b", [(0, 0), (-1, -1), (1 << 32, 1 << 32), (-(1 << 63), 5), (7, -(1 << 63))])
def test_every_bit_of_key_and_counter_counts(a, b):
    n, rng = 5000, key(a, b)
    x, y = torch.ones(n, dtype=BF, device="cuda"), unwritten(n)
    coat.coat_dropout(x, 0.5, rng, y)
    assert torch.equal(y, want(x, 0.5, rng)[0].to(BF))


def test_share_of_dropped_elements():
    """Of n independent draws a share p is dropped, within six standard deviations; two offsets agree in as many as chance has."""
    n, p = 1 << 22, 0.1
    x = torch.ones(n, dtype=BF, device="cuda")
    masks = []
    for offset in (0, 1):
        y = unwritten(n)
        coat.coat_dropout(x, p, key(9, offset), y)
        masks.append(y != 0)
        assert abs((~masks[-1]).double().mean().item() - p) <= 6 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -17
    both = (~masks[0] & ~masks[1]).double().mean().item()
    assert abs(both - p * p) <= 6 * (p * p * (1 - p * p) / n) ** 0.5 + 2.0 ** -17


def test_dropped_elements_do_not_count():
    n, p, rng = 4096, 0.3, key(5, 6)
    keep = want(torch.ones(n, device="cuda"), p, rng)[1]
    for bad in (float("nan"), float("inf")):
        x = torch.where(keep, torch.ones(n, device="cuda"), torch.full((n,), bad, device="cuda")).to(BF)
        y = unwritten(n)
        coat.coat_dropout(x, p, rng, y, residual=torch.zeros_like(x))
        assert y.isfinite().all() and not y[~keep].any()
        coat.coat_dropout_backward(x, p, rng, y)
        assert y.isfinite().all() and not y[~keep].any()


@pytest.mark.parametrize("shift", [8, 16])
def test_pointers_of_16_bytes(shift):
    n, rng = 1003, key(1, 2)
    x, r, y = (torch.empty(n + shift, dtype=BF, device="cuda")[shift:] for _ in range(3))
    x.copy_(randn(n, seed=1)), r.copy_(randn(n, seed=2))
    z = unwritten(n)
    coat.coat_dropout(x, 0.2, rng, y, residual=r)
    coat.coat_dropout(x.clone(), 0.2, rng, z, residual=r.clone())
    assert torch.equal(y, z)


def test_elements_past_2_31():
    n, rng = (1 << 31) + 1003, key(3, 4)
    x, y = torch.ones(n, dtype=BF, device="cuda"), torch.empty(n, dtype=BF, device="cuda")
    coat.coat_dropout(x, 0.25, rng, y)
    for start in (0, (1 << 31) - 500, n - 700):
        assert torch.equal(y[start:start + 700], want(x[start:start + 700], 0.25, rng, start)[0].to(BF))


def test_a_captured_graph_draws_anew_once_rng_has_changed():
    n, rng = 3000, key(1, 0)
    x, y, dx = randn(n, seed=1).to(BF), unwritten(n), unwritten(n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        coat.coat_dropout(x, 0.4, rng, y)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        coat.coat_dropout(x, 0.4, rng, y)
        coat.coat_dropout_backward(y, 0.4, rng, dx)
        rng[1] += 1
    kept = []
    for i in range(3):
        before = rng.clone()
        graph.replay()
        torch.cuda.synchronize()
        ref, keep, size = want(x, 0.4, before)
        near(y, ref, bf16_bound(ref) + 2 * E * size, "y")
        assert torch.equal(dx != 0, keep & (x != 0)) and rng[1].item() == before[1].item() + 1
        kept.append(keep)
    assert not torch.equal(kept[0], kept[1]) and not torch.equal(kept[1], kept[2])


def test_differences():
    """Linear in x with one mask: <dy, y(x + t) - y(x)> = <dx(dy), t>; p = 1/2, whose scale is 2: everything is exact."""
    n, rng = 4000, key(8, 8)
    x, t, dy = (torch.randint(-8, 9, (n,), device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(BF) for i in range(3))
    a, b, dx = unwritten(n), unwritten(n), unwritten(n)
    coat.coat_dropout(x, 0.5, rng, a)
    coat.coat_dropout(x + t, 0.5, rng, b)
    coat.coat_dropout_backward(dy, 0.5, rng, dx)
    assert (dy.double() * (b.double() - a.double())).sum() == (dx.double() * t.double()).sum()


def test_refusals():
    x, rng = torch.zeros(64, dtype=BF, device="cuda"), key(0, 0)
    y = torch.zeros_like(x)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(coat.CoatError, match="INVALID_ARG"):
            coat.coat_dropout(x, p, rng, y)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_dropout(x, 0.1, rng, x)
    with pytest.raises(TypeError, match="rng"):
        coat.coat_dropout(x, 0.1, rng.int(), y)
    with pytest.raises(ValueError, match="rng"):
        coat.coat_dropout(x, 0.1, rng[:1], y)
    with pytest.raises(ValueError, match="rng"):
        coat.coat_dropout(x, 0.1, rng.cpu(), y)
    with pytest.raises(ValueError, match="residual"):
        coat.coat_dropout(x, 0.1, rng, y, residual=y[:32])
    with pytest.raises(ValueError, match="contiguous"):
        coat.coat_dropout_backward(torch.zeros(64, 2, dtype=BF, device="cuda")[:, 0], 0.1, rng, y)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 65535])
def test_the_threshold_is_rounded_up_from_the_middle(T):
    """p = (T - 1/2) / 65536, which float32 holds: draws of T - 1 are dropped, draws of T kept.  Of 2^22 draws 64 are one value, in the
    mean."""
    n, rng = 1 << 22, key(21, T)
    x, y = torch.ones(n, dtype=BF, device="cuda"), unwritten(n)
    coat.coat_dropout(x, (T - 0.5) / 65536, rng, y)
    d = draws(rng.tolist(), 0, n).cuda()
    assert (d == T - 1).any() and (d == T).any()
    assert torch.equal(y != 0, d >= T)
