"""The example's training step on the GPU: its gradients against automatic
differentiation of the same decoder in float64, and a loss that falls.

Bounds: a checkpoint's value is off by 2^-4 of itself at most, 2^-4 / sqrt(12)
in the mean square of evenly spread quotients between two steps (a step is 2^-3
to 2^-4 of the value), so 0.02 to 0.04; bf16 adds 2^-9 at each of a dozen
roundings along the way.  A gradient's relative error in the l2 norm is then a
few of these added in squares, since the errors of different entries do not
line up: 1/8 leaves a factor of three.  A wrong factor, sign, index or missing
term is an error of the order of one.  The forward pass has no 8-bit values: its
loss is within 2^-5.
"""
import pathlib
import sys

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu
sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1] / "examples"))


def _reference(model, ids, targets):
    """Loss and gradients in float64 from the weights that the step multiplies with."""
    cfg, M = model.cfg, model.M
    w = {n: (model.w[n] if model.w[n].dim() == 1 else model.w16[n]).double().requires_grad_() for n in model.w}
    Hq, Hk, D = cfg.heads, cfg.kv_heads, cfg.head_dim
    c, s = (t[model.positions.long()].double()[:, None] for t in (model.cos, model.sin))

    def norm(x, weight):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + cfg.eps) * weight

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    h = w["embed"][ids]
    for i in range(cfg.layers):
        qkv = (norm(h, w[f"norm1.{i}"]) @ w[f"qkv.{i}"].T).view(M, Hq + 2 * Hk, D)
        q, k, v = qkv.split((Hq, Hk, Hk), 1)
        q, k = turn(norm(q, w[f"q_norm.{i}"])), turn(norm(k, w[f"k_norm.{i}"]))
        q, k, v = (t.view(M // cfg.seq, cfg.seq, -1, D).transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
        scores = (q @ k.transpose(-1, -2) / D ** 0.5).masked_fill(
            torch.ones(cfg.seq, cfg.seq, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        o = (scores.softmax(-1) @ v).transpose(1, 2).reshape(M, -1)
        h = h + o @ w[f"out.{i}"].T
        gate, up = (norm(h, w[f"norm2.{i}"]) @ w[f"gate_up.{i}"].T).chunk(2, -1)
        h = h + (F.silu(gate) * up) @ w[f"down.{i}"].T
    loss = F.cross_entropy(norm(h, w["norm"]) @ w["head"].T, targets)
    loss.backward()
    return loss.item(), {n: t.grad for n, t in w.items()}


@pytest.fixture(scope="module")
def example():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    import train_decoder
    return train_decoder


@pytest.mark.parametrize("sizes", [dict(layers=2, width=256, heads=4, kv_heads=2, hidden=688, vocab=64, seq=32, group=16),
                                   dict(layers=1, width=384, heads=3, kv_heads=1, hidden=1024, vocab=136, seq=50, group=128)])
def test_gradients(example, sizes):
    cfg = example.Config(**sizes)
    model = example.Decoder(cfg, 4 * cfg.seq)
    ids, targets = example.batch(cfg, model.M, 1)
    model.grad.fill_(float("nan"))
    loss = model.loss_and_gradients(ids, targets)
    want, grads = _reference(model, ids, targets)
    assert abs(loss.item() - want) <= 2.0 ** -5 * want
    for name, ref in grads.items():
        err = (model.g[name].double() - ref).norm() / ref.norm()
        assert err <= 0.125, f"{name}: relative error {err:.3f}"


def test_loss_falls(example):
    cfg = example.Config(layers=2, width=256, heads=4, kv_heads=2, hidden=688, vocab=64, seq=64, group=16)
    model = example.Decoder(cfg, 1024)
    losses = [model.step(*example.batch(cfg, model.M, 7), lr=3e-3).item() for _ in range(30)]
    assert losses[-1] < 0.5 * losses[0], losses
