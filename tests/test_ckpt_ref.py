"""The float64 forms that the checkpointing operators are tested against: their
gradients against central differences and autograd, their quantizer against the
oracle (CPU only)."""
import numpy as np
import pytest
import torch

import _ckpt_ref as R
import oracle
from coat_fp8_adamw_gb300 import synth


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _differences(f, x, d, h=1e-5):
    """Central differences of sum(f(x) d) in every entry of x (error h^2 f''' / 6 + 2^-53 / h: about 1e-10 here)."""
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = (f(x) * d).sum()
        flat[i] = keep - h
        down = (f(x) * d).sum()
        flat[i] = keep
        o[i] = (up - down) / (2 * h)
    return out


def test_norm_gradient_against_differences():
    x = torch.randn(3, 16, generator=_gen(0), dtype=torch.float64)
    w = 1 + 0.1 * torch.randn(16, generator=_gen(1), dtype=torch.float64)
    dy = torch.randn(3, 16, generator=_gen(2), dtype=torch.float64)
    eps = 1e-2
    dx, dw, _, _ = R.rmsnorm_backward(dy, x, R.rmsnorm(x, w, eps)[1], w)
    assert torch.allclose(dx, _differences(lambda t: R.rmsnorm(t, w, eps)[0], x, dy), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda t: R.rmsnorm(x, t, eps)[0], w, dy), atol=1e-8)


def test_swiglu_gradient_against_differences():
    g = 3 * torch.randn(2, 16, generator=_gen(3), dtype=torch.float64)
    u = torch.randn(2, 16, generator=_gen(4), dtype=torch.float64)
    d = torch.randn(2, 16, generator=_gen(5), dtype=torch.float64)
    dg, du = R.swiglu_backward(d, g, u)
    assert torch.allclose(dg, _differences(lambda t: R.swiglu(t, u), g, d), atol=1e-8)
    assert torch.allclose(du, _differences(lambda t: R.swiglu(g, t), u, d), atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32])
def test_qk_gradient_against_differences(rot, interleaved):
    x = torch.randn(2, 2, 32, generator=_gen(6), dtype=torch.float64)
    w = 1 + 0.1 * torch.randn(32, generator=_gen(7), dtype=torch.float64)
    d = torch.randn(2, 2, 32, generator=_gen(8), dtype=torch.float64)
    a = torch.rand(2, rot // 2, generator=_gen(9), dtype=torch.float64) * 6
    c, s = a.cos(), a.sin()
    f = lambda t, v: R.qk(t, v, 1e-2, c, s, rot, interleaved)[0]  # noqa: E731
    dx, dw, _, _ = R.qk_backward(d, x, R.qk(x, w, 1e-2, c, s, rot, interleaved)[1], w, c, s, rot, interleaved)
    assert torch.allclose(dx, _differences(lambda t: f(t, w), x, d), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda t: f(x, t), w, d), atol=1e-8)
    # a rotation keeps lengths, and the back turn undoes it
    y = R.rotate(x, c, s, rot, interleaved)
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1))
    assert torch.allclose(R.rotate(y, c, -s, rot, interleaved), x)


def test_weight_gradient_is_autograds():
    x = torch.randn(7, 16, generator=_gen(10), dtype=torch.float64)
    W = torch.randn(8, 16, generator=_gen(11), dtype=torch.float64, requires_grad=True)
    dy = torch.randn(7, 8, generator=_gen(12), dtype=torch.float64)
    r, c = torch.rand(7, generator=_gen(13), dtype=torch.float64), torch.rand(16, generator=_gen(14), dtype=torch.float64)
    ((x * r[:, None] * c) @ W.T * dy).sum().backward()
    assert torch.allclose(R.weight_grad(dy, x, r, c)[0], W.grad)


@pytest.mark.parametrize("G", [8, 32, 128])
def test_quantizer_is_the_oracles(G):
    rng = np.random.default_rng(G)
    x = rng.standard_normal((16, 256)) * 10.0 ** rng.uniform(-4, 4, (16, 1))
    x[3] = 0
    bits = synth.f32_to_bf16_bits(x.astype(np.float32)).reshape(x.shape)
    q, _, S = oracle.act_quantize(bits, G)
    val, Sr, _ = R.quantize(torch.from_numpy(synth.bf16_bits_to_f32(bits)).double(), G)
    assert np.array_equal(Sr.numpy().astype(np.float32), S.reshape(Sr.shape))
    dec = torch.from_numpy(q).view(torch.float8_e4m3fn).double()
    assert torch.equal(val, dec)
