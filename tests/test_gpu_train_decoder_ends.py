"""The example's training step with dropout, a tied table and tokens without a target: its gradients against automatic
differentiation of the same decoder in float64, with the masks that the generator's definition gives.

The bound is that of the example's other gradients: the 8-bit checkpoints are off by 0.02 to 0.04 in the mean square, a few of
these added in squares; 1/8 leaves a factor of three.  The tied table's gradient has the output layer's part, from bf16 values
alone, and the embedding's.  A mask that is another one backward than forward, a missing or doubled part of the tied gradient
or a counted token without a target is an error of the order of one."""
import pathlib
import sys

import pytest
import torch
import torch.nn.functional as F

from _lm_ref import draws, threshold

pytestmark = pytest.mark.gpu
sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1] / "examples"))


@pytest.fixture(scope="module")
def example():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    import train_decoder
    return train_decoder


def _reference(model, ids, targets, rng):
    """Loss and gradients in float64 from the weights that the step multiplies with."""
    cfg, M = model.cfg, model.M
    w = {n: (model.w[n] if model.w[n].dim() == 1 else model.w16[n]).double().requires_grad_() for n in model.w}
    Hq, Hk, D = cfg.heads, cfg.kv_heads, cfg.head_dim
    c, s = (t[model.positions.long()].double()[:, None] for t in (model.cos, model.sin))
    T = threshold(cfg.dropout)

    def norm(x, weight):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + cfg.eps) * weight

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def drop(x, place):
        keep = (draws(rng[place].tolist(), 0, x.numel()) >= T).view(x.shape).cuda()
        return torch.where(keep, x * (65536 / (65536 - T)), 0.0)

    h = torch.where((ids >= 0)[:, None], w["embed"][ids.clamp_min(0)], 0.0)
    for i in range(cfg.layers):
        qkv = (norm(h, w[f"norm1.{i}"]) @ w[f"qkv.{i}"].T).view(M, Hq + 2 * Hk, D)
        q, k, v = qkv.split((Hq, Hk, Hk), 1)
        q, k = turn(norm(q, w[f"q_norm.{i}"])), turn(norm(k, w[f"k_norm.{i}"]))
        q, k, v = (t.view(M // cfg.seq, cfg.seq, -1, D).transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
        scores = (q @ k.transpose(-1, -2) / D ** 0.5).masked_fill(
            torch.ones(cfg.seq, cfg.seq, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        o = (scores.softmax(-1) @ v).transpose(1, 2).reshape(M, -1)
        h = h + drop(o @ w[f"out.{i}"].T, 2 * i)
        gate, up = (norm(h, w[f"norm2.{i}"]) @ w[f"gate_up.{i}"].T).chunk(2, -1)
        h = h + drop((F.silu(gate) * up) @ w[f"down.{i}"].T, 2 * i + 1)
    loss = F.cross_entropy(norm(h, w["norm"]) @ w[cfg.head].T, targets, ignore_index=-100)
    loss.backward()
    return loss.item(), {n: t.grad for n, t in w.items()}


@pytest.mark.parametrize("dropout,tied,index", [(0.25, True, torch.int64), (0.1, False, torch.int32), (0.0, True, torch.int64)])
def test_gradients(example, dropout, tied, index):
    cfg = example.Config(layers=2, width=256, heads=4, kv_heads=2, hidden=688, vocab=200, seq=40, group=16, dropout=dropout, tied=tied)
    model = example.Decoder(cfg, 4 * cfg.seq, seed=3)
    ids, targets = example.batch(cfg, model.M, 1)
    targets[::7] = -100
    model.grad.fill_(float("nan"))
    rng = model.rng.clone()
    loss = model.loss_and_gradients(ids.to(index), targets.to(index))
    want, grads = _reference(model, ids, targets, rng)
    assert abs(loss.item() - want) <= 2.0 ** -5 * want
    for name, ref in grads.items():
        err = (model.g[name].double() - ref).norm() / ref.norm()
        assert err <= 0.125, f"{name}: relative error {err:.3f}"


def test_masks_change_from_step_to_step_and_not_within_one(example):
    cfg = example.Config(layers=1, width=256, heads=4, kv_heads=2, hidden=688, vocab=64, seq=32, group=16, dropout=0.3)
    model = example.Decoder(cfg, 128)
    ids, targets = example.batch(cfg, model.M, 1)
    first, again = model.loss_and_gradients(ids, targets).item(), model.loss_and_gradients(ids, targets).item()
    assert first == again
    before = model.rng.clone()
    model.step(ids, targets, lr=0.0)
    assert torch.equal(model.rng[:, 1], before[:, 1] + len(before)) and torch.equal(model.rng[:, 0], before[:, 0])
    assert len(set(torch.cat((before, model.rng))[:, 1].tolist())) == 2 * len(before)


@pytest.mark.parametrize("tied", [False, True])
def test_a_batch_without_a_target(example, tied):
    """Padding alone: loss 0 and zero gradients, and the optimizer's step leaves numbers."""
    cfg = example.Config(layers=1, width=256, heads=4, kv_heads=2, hidden=688, vocab=64, seq=32, group=16, dropout=0.1, tied=tied)
    model = example.Decoder(cfg, 128)
    ids, targets = example.batch(cfg, model.M, 1)
    targets.fill_(-100)
    model.grad.fill_(float("nan"))
    assert model.loss_and_gradients(ids, targets).item() == 0.0 and not model.grad.any()
    model.step(ids, targets)
    assert model.flat.isfinite().all()
