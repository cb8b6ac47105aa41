"""Training of a small decoder on activations kept in 8 bits.

One training step as the operators are meant to be used together: every norm,
the heads' norm with its rotation and the gated unit leave an 8-bit checkpoint of
what went into them; the backward pass reads the checkpoints alone, writes the
weight gradients (coat_ckpt_weight_grad) and the norms' gradients into one flat
bf16 gradient, and coat_fp8_adamw_step updates all parameters from it in one
call.  Projections' outputs and input gradients are torch matrix products, and
attention is torch's, which keeps its own inputs (q, k, v) in bf16.

    python examples/train_decoder.py [--layers 4] [--width 1024] [--tokens 2048] [--steps 20]
"""
from __future__ import annotations

import argparse
import math
import pathlib
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
import coat_fp8_adamw_gb300 as coat  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Config:
    def __init__(self, layers=4, width=1024, heads=8, kv_heads=2, hidden=2816, vocab=512, seq=256, group=128, eps=1e-5):
        self.layers, self.width, self.heads, self.kv_heads, self.hidden = layers, width, heads, kv_heads, hidden
        self.vocab, self.seq, self.group, self.eps = vocab, seq, group, eps
        self.head_dim = width // heads
        self.head_group = min(group, self.head_dim)

    def shapes(self):
        C, D, qkv = self.width, self.head_dim, (self.heads + 2 * self.kv_heads) * self.head_dim
        block = [("norm1", (C,)), ("qkv", (qkv, C)), ("q_norm", (D,)), ("k_norm", (D,)), ("out", (C, self.heads * D)),
                 ("norm2", (C,)), ("gate_up", (2 * self.hidden, C)), ("down", (C, self.hidden))]
        return ([("embed", (self.vocab, C))] + [(f"{n}.{i}", s) for i in range(self.layers) for n, s in block]
                + [("norm", (C,)), ("head", (self.vocab, C))])


def views(flat, shapes):
    """One view per parameter; every one starts on 16 bytes, since all sizes are multiples of 16."""
    out, at = {}, 0
    for name, shape in shapes:
        n = math.prod(shape)
        out[name] = flat[at:at + n].view(shape)
        at += n
    return out


class Checkpoint:
    """An activation in 8 bits: codes and one scale per group (and, behind a norm, 1/rms of every row)."""

    def __init__(self, shape, G, rows=None):
        self.q = torch.empty(shape, dtype=U8, device="cuda")
        self.scale = torch.empty((*shape[:-1], shape[-1] // G), dtype=F32, device="cuda")
        self.rstd = None if rows is None else torch.empty(rows, dtype=F32, device="cuda")
        self.G = G

    def bytes(self):
        return sum(t.numel() * t.element_size() for t in (self.q, self.scale, self.rstd) if t is not None)


class Decoder:
    def __init__(self, cfg: Config, tokens: int, seed=0):
        self.cfg, self.M = cfg, tokens
        shapes = cfg.shapes()
        n = sum(math.prod(s) for _, s in shapes)
        self.flat = torch.empty(n, device="cuda")
        self.w = views(self.flat, shapes)
        g = torch.Generator(device="cuda").manual_seed(seed)
        for name, shape in shapes:
            if len(shape) == 1:
                self.w[name].fill_(1.0)
            else:
                self.w[name].normal_(0.0, 0.02 if name == "embed" else shape[1] ** -0.5, generator=g)
        self.flat16, self.grad = self.flat.to(BF), torch.zeros(n, dtype=BF, device="cuda")
        self.w16, self.g = views(self.flat16, shapes), views(self.grad, shapes)
        self.m_q, self.v_q = (torch.zeros(n, dtype=U8, device="cuda") for _ in range(2))
        self.meta = torch.tensor([0.0, 1.0, 0.0, 1.0], device="cuda").repeat(coat.num_groups(n, 128), 1)
        self.steps = 0
        D = cfg.head_dim
        angle = torch.arange(cfg.seq, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.positions = (torch.arange(tokens, device="cuda") % cfg.seq).to(torch.int32)
        need = max([coat.coat_rmsnorm_ckpt_backward_workspace_bytes(tokens, cfg.width),
                    coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(tokens, D)]
                   + [coat.coat_ckpt_weight_grad_workspace_bytes(tokens, *s) for _, s in shapes if len(s) == 2])
        self.workspace = torch.empty(max(need, 16), dtype=U8, device="cuda")

    def new(self, *shape):
        return torch.empty(shape, dtype=BF, device="cuda")

    def norm(self, x, residual, weight):
        """y, h = x + residual, and h's checkpoint."""
        c = Checkpoint(x.shape, self.cfg.group, self.M)
        y, h = torch.empty_like(x), x if residual is None else torch.empty_like(x)
        coat.coat_rmsnorm_ckpt(x, weight, self.cfg.eps, c.G, y, c.q, c.scale, c.rstd, residual=residual,
                               h=None if residual is None else h)
        return y, h, c

    def attention(self, q, k, v):
        cfg, B = self.cfg, self.M // self.cfg.seq
        q, k, v = (t.view(B, cfg.seq, -1, cfg.head_dim).transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(cfg.heads // cfg.kv_heads, 1) for t in (k, v))
        return F.scaled_dot_product_attention(q, k, v, is_causal=True).transpose(1, 2).reshape(self.M, -1)

    def forward(self, ids):
        cfg, w, M, D = self.cfg, self.w16, self.M, self.cfg.head_dim
        Hq, Hk = cfg.heads, cfg.kv_heads
        x, delta, kept = w["embed"][ids], None, []
        for i in range(cfg.layers):
            y, h, c1 = self.norm(x, delta, self.w[f"norm1.{i}"])
            qkv = (y @ w[f"qkv.{i}"].T).view(M, Hq + 2 * Hk, D)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:].contiguous()
            cq, ck = (Checkpoint((M, H, D), cfg.head_group, (M, H)) for H in (Hq, Hk))
            qr, kr = self.new(M, Hq, D), self.new(M, Hk, D)
            coat.coat_qk_norm_rope_ckpt(q, k, self.w[f"q_norm.{i}"], self.w[f"k_norm.{i}"], cfg.eps, self.cos, self.sin,
                                        self.positions, cq.G, qr, cq.q, cq.scale, cq.rstd, kr, ck.q, ck.scale, ck.rstd)
            o = self.attention(qr, kr, v)
            padded = F.pad(o, (0, 0, 0, -M % 16))          # this quantizer takes 16 rows at a time
            co = Checkpoint(padded.shape, cfg.group)
            coat.coat_act_quantize_fp8(padded, co.G, co.q, co.scale)
            co.q, co.scale = co.q[:M], co.scale[:M]
            y, h, c2 = self.norm(o @ w[f"out.{i}"].T, h, self.w[f"norm2.{i}"])
            both = y @ w[f"gate_up.{i}"].T
            a = self.new(M, cfg.hidden)
            cg, cu = (Checkpoint(a.shape, cfg.group) for _ in range(2))
            coat.coat_swiglu_ckpt(both[:, :cfg.hidden], both[:, cfg.hidden:], cg.G, a, cg.q, cg.scale, cu.q, cu.scale)
            x, delta = h, a @ w[f"down.{i}"].T
            kept.append((c1, cq, ck, (qr, kr, v), co, c2, cg, cu))
        y, _, c = self.norm(x, delta, self.w["norm"])
        return y @ w["head"].T, kept, c

    def weight_grad(self, name, dy, c, norm_weight=None):
        """Behind a norm the checkpoint is of the norm's input: 1/rms and the weight make it its output."""
        coat.coat_ckpt_weight_grad(dy, c.q, c.scale, c.G, self.g[name], self.workspace,
                                   row_scale=None if norm_weight is None else c.rstd, col_scale=norm_weight)

    def norm_backward(self, name, dy, c, dresidual=None):
        dx = torch.empty_like(dy)
        coat.coat_rmsnorm_ckpt_backward(dy, c.q, c.scale, c.rstd, self.w[name], c.G, dx, self.g[name], self.workspace,
                                        dresidual=dresidual)
        return dx

    def backward(self, ids, dlogits, kept, last):
        cfg, w, M, D = self.cfg, self.w16, self.M, self.cfg.head_dim
        Hq, Hk = cfg.heads, cfg.kv_heads
        self.weight_grad("head", dlogits, last, self.w["norm"])
        d = self.norm_backward("norm", dlogits @ w["head"], last)
        for i in reversed(range(cfg.layers)):
            c1, cq, ck, qkv, co, c2, cg, cu = kept.pop()
            da = d @ w[f"down.{i}"]
            dboth, ca = self.new(M, 2 * cfg.hidden), Checkpoint(da.shape, cfg.group)
            coat.coat_swiglu_ckpt_backward(da, cg.q, cg.scale, cu.q, cu.scale, cg.G, dboth[:, :cfg.hidden],
                                           dboth[:, cfg.hidden:], h_q=ca.q, h_scale=ca.scale)
            self.weight_grad(f"down.{i}", d, ca)
            self.weight_grad(f"gate_up.{i}", dboth, c2, self.w[f"norm2.{i}"])
            d = self.norm_backward(f"norm2.{i}", dboth @ w[f"gate_up.{i}"], c2, d)
            self.weight_grad(f"out.{i}", d, co)
            do = d @ w[f"out.{i}"]
            with torch.enable_grad():
                leaves = [t.detach().requires_grad_() for t in qkv]
                dqr, dkr, dv = torch.autograd.grad(self.attention(*leaves), leaves, do)
            dqkv = self.new(M, Hq + 2 * Hk, D)
            dqkv[:, Hq + Hk:] = dv
            coat.coat_qk_norm_rope_ckpt_backward(dqr.contiguous(), dkr.contiguous(), cq.q, cq.scale, cq.rstd, ck.q, ck.scale,
                                                 ck.rstd, self.w[f"q_norm.{i}"], self.w[f"k_norm.{i}"], self.cos, self.sin,
                                                 self.positions, cq.G, dqkv[:, :Hq], dqkv[:, Hq:Hq + Hk],
                                                 self.g[f"q_norm.{i}"], self.g[f"k_norm.{i}"], self.workspace)
            dqkv = dqkv.view(M, -1)
            self.weight_grad(f"qkv.{i}", dqkv, c1, self.w[f"norm1.{i}"])
            d = self.norm_backward(f"norm1.{i}", dqkv @ w[f"qkv.{i}"], c1, d)
        self.g["embed"].copy_(torch.zeros(cfg.vocab, cfg.width, device="cuda").index_add_(0, ids, d.float()))

    @torch.no_grad()
    def loss_and_gradients(self, ids, targets):
        logits, kept, last = self.forward(ids)
        logp = F.log_softmax(logits.float(), -1)
        loss = F.nll_loss(logp, targets)
        self.kept_bytes = sum(c.bytes() for block in kept for c in block if isinstance(c, Checkpoint)) + last.bytes()
        dlogits = logp.exp()
        dlogits[torch.arange(self.M, device="cuda"), targets] -= 1
        self.backward(ids, (dlogits / self.M).to(BF), kept, last)
        return loss

    def step(self, ids, targets, lr=1e-3):
        loss = self.loss_and_gradients(ids, targets)
        self.steps += 1
        coat.coat_fp8_adamw_step(self.flat, self.grad, self.m_q, self.v_q, self.meta, 128, 0.9, 0.95, lr, 1e-8, 0.1, self.steps)
        self.flat16.copy_(self.flat)
        return loss


def batch(cfg, tokens, seed):
    """Sequences in which a token and its predecessor decide the next one."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randint(0, cfg.vocab, (tokens // cfg.seq, cfg.seq + 1), generator=g)
    for t in range(2, cfg.seq + 1):
        s[:, t] = (s[:, t - 1] + s[:, t - 2]) % 61
    s = s.cuda()
    return s[:, :-1].reshape(-1), s[:, 1:].reshape(-1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    cfg = Config(layers=a.layers, width=a.width)
    model = Decoder(cfg, a.tokens)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(a.steps):
        ids, targets = batch(cfg, a.tokens, i)
        begin.record()
        loss = model.step(ids, targets)
        end.record()
        print(f"step {i + 1:3d}  loss {loss.item():.4f}  {begin.elapsed_time(end):.2f} ms", flush=True)
    print(f"activations kept in 8 bits: {model.kept_bytes / a.tokens:.0f} bytes a token")


if __name__ == "__main__":
    main()
