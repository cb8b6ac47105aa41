"""The operators with 8-bit activation checkpoints on the GPU, through the
binding, against their float64 forms.

Bounds, per element (u = 2^-8: half a bf16 step, relatively; e = 2^-24):
  * a bf16 output is its float32 value rounded once: u |ref| (1 + u) plus the
    float32 value's own error;
  * a row's sum of squares adds N positive terms in a tree of at most
    16 + 10 + 2 levels per thread, warp and block, so 1/rms is within 20 e and
    y = x rstd w within 24 e, relatively: 2^-19 covers it;
  * dx: g, xh and c are within a few e of exact ones and c within 40 e of
    mean|g xh|; the differences cancel, so the bound is 2^-18 of the sizes of
    the terms, r (|g| + |xh| mean|g xh|);
  * dw adds M terms (M H for heads): (M + 64) e sum|terms|;
  * silu: the argument of the exponential is rounded (|g| e), the exponential and
    the quotient are within 4 e: (|g| + 8) 2 e; below 2^-120 it may be flushed;
  * the weight gradient's operand is rounded to bf16 (u) and added in float32
    on M terms, truncating at worst: u + (M + 8) 2^-22 of sum|dy x|;
  * codes and scales of bf16 inputs are exact; those of silu(gate) up, whose
    float32 value carries silu's error, are within it plus half a grid step.
"""
import math

import pytest
import torch

import _ckpt_ref as R
import coat_fp8_adamw_gb300 as coat

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
EPS = 1e-5
E4M3 = torch.float8_e4m3fn
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    coat.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def acts(M, N, seed, spread=2.0):
    """Rows of very different sizes, a zero row, a zero group, outliers."""
    x = torch.randn(M, N, generator=gen(seed), device="cuda")
    x *= torch.exp(spread * torch.randn(M, 1, generator=gen(seed + 1), device="cuda"))
    x[torch.rand(M, N, generator=gen(seed + 2), device="cuda") < 1e-3] *= 100
    if M > 2:
        x[1] = 0
        x[2, :min(N, 128)] = 0
    return x.to(BF)


def grads(M, N, seed):
    g = 1e-3 * torch.randn(M, N, generator=gen(seed), device="cuda") * torch.exp(
        torch.randn(M, 1, generator=gen(seed + 1), device="cuda"))
    if M > 3:
        g[3] = 0
    return g.to(BF)


def norm_w(N, seed):
    return 1 + 0.2 * torch.randn(N, generator=gen(seed), device="cuda")


def empty(*shape, dtype=BF):
    """Filled with a value that no result has, so that what is not written shows."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.fill_(0xFF) if dtype == U8 else t.fill_(float("nan"))


def workspace(n):
    return torch.full((max(int(n), 16),), 0xFF, dtype=U8, device="cuda")


def near(got, ref, bound, what):
    got, bad = got.double(), None
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    bad = over.max().item()
    assert bad <= 0, f"{what}: {bad:.3e} over the bound at {int(over.argmax())} (ref {ref.flatten()[over.argmax()]:.6e})"


def bf16_bound(ref):
    return U * (1 + U) * ref.abs() + 2.0 ** -133


def checkpoint(x, G):
    """The checkpoint of bf16 x (its scales exact) as the library holds it, and its values in float64."""
    val, S, _ = R.quantize(x.double(), G)
    q = val.float().to(E4M3)
    q = torch.where(val == 0, torch.zeros_like(val).to(U8), q.view(U8))
    return q, S.float(), R.dequantize(val, S, G)


def check_checkpoint(q, S, x, G, what):
    val, Sr, _ = R.quantize(x.double(), G)
    assert torch.equal(S.double().view(Sr.shape), Sr), f"{what}: scales"
    assert torch.equal(q.view(E4M3).double().view(val.shape), val), f"{what}: codes"
    assert not (q == 0x80).any(), f"{what}: a negative zero"


NORMS = [(1, 16, 8, False), (1, 4096, 128, True), (3, 48, 16, False), (7, 512, 8, True), (5, 528, 16, False),
         (257, 1024, 32, True), (33, 2048, 64, False), (1000, 4096, 128, True), (65, 5120, 128, False), (311, 11008, 32, True),
         (9, 16384, 128, True), (2, 16368, 16, False), (4099, 256, 64, True)]


@pytest.mark.parametrize("M,N,G,res", NORMS)
def test_norm_forward(M, N, G, res):
    x, w = acts(M, N, M + N), norm_w(N, 5)
    r = acts(M, N, M + N + 7) if res else None
    h = empty(M, N) if res else None
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, rstd, residual=r, h=h)
    src = (x.float() + r.float()).to(BF) if res else x
    if res:
        assert torch.equal(h, src)
    ref, rr = R.rmsnorm(src.double(), w.double(), EPS)
    near(rstd, rr, 2.0 ** -19 * rr, "rstd")
    near(y, ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), "y")
    check_checkpoint(q, S, src, G, "checkpoint")


@pytest.mark.parametrize("M,N,G,res", NORMS)
def test_norm_backward(M, N, G, res):
    x, w, dy = acts(M, N, M * N), norm_w(N, 6), grads(M, N, M + 3)
    q, S, xv = checkpoint(x, G)
    rstd = R.rmsnorm(x.double(), w.double(), EPS)[1].float()
    dres = grads(M, N, M + 4) if res else None
    dx, dw = empty(M, N), empty(N)
    ws = workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N))
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw, ws, dresidual=dres)
    rx, rw, sx, sw = R.rmsnorm_backward(dy.double(), xv, rstd.double(), w.double())
    if res:
        rx = rx + dres.double()
    near(dx, rx, bf16_bound(rx) + 2.0 ** -18 * sx + 2 * E * rx.abs(), "dx")
    near(dw, rw, bf16_bound(rw) + (M + 64) * E * sw, "dweight")
    dx2, dw2 = empty(M, N), empty(N)
    ws.fill_(0x7F)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx2, dw2, ws, dresidual=dres)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2), "two calls differ"


def silu_bound(ref, g):
    return (g.abs() + 8) * 2 * E * ref.abs() + 2.0 ** -120 * g.abs()


SWIGLU = [(1, 16, 8, False), (1, 8192, 16, True), (3, 48, 16, True), (17, 8192, 128, False), (129, 272, 16, True),
          (515, 1376, 32, True), (64, 13824, 128, False), (2049, 128, 64, True)]


@pytest.mark.parametrize("M,N,G,fused", SWIGLU)
def test_swiglu_forward(M, N, G, fused):
    both = acts(M, 2 * N + 24, M + N)
    g, u = (both[:, 8:N + 8], both[:, N + 16:2 * N + 16]) if fused else (both[:, :N].contiguous(), both[:, N:2 * N].contiguous())
    h = empty(M, N)
    gq, uq = empty(M, N, dtype=U8), empty(M, N, dtype=U8)
    gs, us = empty(M, N // G, dtype=F32), empty(M, N // G, dtype=F32)
    coat.coat_swiglu_ckpt(g, u, G, h, gq, gs, uq, us)
    G64, U64 = g.double(), u.double()
    ref = R.swiglu(G64, U64)
    near(h, ref, bf16_bound(ref) + silu_bound(ref, G64) + 2.0 ** -120 * (G64 * U64).abs(), "h")
    check_checkpoint(gq, gs, g, G, "gate")
    check_checkpoint(uq, us, u, G, "up")


@pytest.mark.parametrize("M,N,G,fused", SWIGLU)
@pytest.mark.parametrize("with_h", [False, True])
def test_swiglu_backward(M, N, G, fused, with_h):
    both, dh = acts(M, 2 * N, M + N + 1), grads(M, N, M)
    (gq, gs, g), (uq, us, u) = checkpoint(both[:, :N], G), checkpoint(both[:, N:], G)
    if fused:
        d = empty(M, 2 * N + 8)
        dg, du = d[:, N + 8:], d[:, :N]
    else:
        dg, du = empty(M, N), empty(M, N)
    hq, hs = (empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)) if with_h else (None, None)
    coat.coat_swiglu_ckpt_backward(dh, gq, gs, uq, us, G, dg, du, h_q=hq, h_scale=hs)
    D = dh.double()
    rg, ru = R.swiglu_backward(D, g, u)
    s = torch.special.expit(g)
    # 1 - s cancels to e of 1, and the two terms of s + g s (1 - s) may cancel
    size = (D * u).abs() * (s + (g * s).abs())
    near(dg, rg, bf16_bound(rg) + (g.abs() + 16) * 4 * E * size + 2.0 ** -120 * (D * u * g).abs(), "dgate")
    near(du, ru, bf16_bound(ru) + silu_bound(ru, g) + 2.0 ** -120 * (D * g).abs(), "dup")
    if fused:
        assert torch.isnan(d[:, N:N + 8]).all(), "written between the two"
    if with_h:
        h = R.swiglu(g, u)
        err = silu_bound(h, g) + 2.0 ** -120 * (g * u).abs()
        Sr = h.unflatten(-1, (-1, G)).abs().amax(-1) / 448
        near(hs, Sr, err.unflatten(-1, (-1, G)).amax(-1) / 448 + 2 * E * Sr + 2.0 ** -140, "h scale")
        S = hs.double().repeat_interleave(G, -1)
        val = hq.view(E4M3).double()
        ratio = torch.where(S > 0, h / torch.where(S > 0, S, 1.0), 0.0)
        half = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp_min(2.0 ** -6) * (1 + 2.0 ** -16))) - 4)
        near(val, ratio, half + torch.where(S > 0, err / torch.where(S > 0, S, 1.0), 0.0) + 2.0 ** -20 * ratio.abs(), "h codes")
        assert not (hq == 0x80).any()


def rope_tables(max_pos, rot):
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    return a.cos().float(), a.sin().float()


# M, Hq, Hk, D, rot, G, interleaved
QK = [(1, 1, 1, 16, 16, 8, False), (1, 1, 0, 16, 16, 16, True), (3, 16, 4, 64, 32, 16, True), (5, 5, 1, 80, 80, 16, False),
      (33, 7, 7, 80, 64, 8, True), (2, 3, 2, 112, 96, 16, False), (129, 32, 8, 128, 128, 128, False), (700, 40, 10, 128, 128, 64, False),
      (64, 4, 4, 256, 256, 128, True), (31, 6, 2, 256, 64, 32, False), (11, 9, 3, 48, 32, 8, False), (1300, 3, 1, 32, 32, 32, False),
      (4, 64, 64, 128, 64, 32, True)]


def qk_inputs(M, Hq, Hk, D, rot, seed):
    qkv = acts(M, (Hq + 2 * Hk) * D, seed)
    q = qkv[:, :Hq * D].view(M, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D) if Hk else None
    max_pos = 97
    cos, sin = rope_tables(max_pos, rot)
    pos = torch.randint(0, max_pos, (M,), generator=gen(seed + 9), device="cuda", dtype=torch.int32)
    pos[0] = max_pos - 1
    return q, k, cos, sin, pos


@pytest.mark.parametrize("M,Hq,Hk,D,rot,G,inter", QK)
def test_qk_forward(M, Hq, Hk, D, rot, G, inter):
    q, k, cos, sin, pos = qk_inputs(M, Hq, Hk, D, rot, M + D)
    ws = [norm_w(D, 1), norm_w(D, 2)]
    outs = [[empty(M, H, D), empty(M, H, D, dtype=U8), empty(M, H, D // G, dtype=F32), empty(M, H, dtype=F32)] for H in (Hq, Hk)]
    coat.coat_qk_norm_rope_ckpt(q, k, ws[0], ws[1] if Hk else None, EPS, cos, sin, pos, G, *outs[0],
                                *(outs[1] if Hk else [None] * 4), interleaved=inter)
    c, s = cos[pos.long()].double(), sin[pos.long()].double()
    for x, w, (y, codes, scale, rstd), what in zip((q, k), ws, outs, "qk"):
        if x is None:
            continue
        ref, rr = R.qk(x.double(), w.double(), EPS, c, s, rot, inter)
        # the two products of a turned pair may cancel
        size = R.rmsnorm(x.double(), w.double(), EPS)[0].abs()
        size = R.rotate(size, c.abs(), -s.abs(), rot, inter).abs() + R.rotate(size, c.abs(), s.abs(), rot, inter).abs()
        near(rstd, rr, 2.0 ** -19 * rr, what + " rstd")
        near(y, ref, bf16_bound(ref) + 2.0 ** -18 * size, what + " out")
        check_checkpoint(codes, scale, x, G, what)


@pytest.mark.parametrize("M,Hq,Hk,D,rot,G,inter", QK)
def test_qk_backward(M, Hq, Hk, D, rot, G, inter):
    q, k, cos, sin, pos = qk_inputs(M, Hq, Hk, D, rot, M + D + 1)
    c, s = cos[pos.long()].double(), sin[pos.long()].double()
    buf = empty(M, (Hq + 2 * Hk) * D + 8)
    sides, args = [], []
    for x, H, seed, start in ((q, Hq, 1, 0), (k, Hk, 2, Hq * D)):
        if x is None:
            args.append([None] * 7)
            continue
        w = norm_w(D, seed)
        codes, scale, xv = checkpoint(x, G)
        rstd = R.rmsnorm(x.double(), w.double(), EPS)[1].float()
        dy = grads(M, H * D, M + seed).view(M, H, D)
        dx, dw = buf[:, start:start + H * D].view(M, H, D), empty(D)
        sides.append((dy, xv, rstd, w, dx, dw))
        args.append([dy, codes, scale, rstd, w, dx, dw])
    (dyq, cq, sq, rq, wq, dq, dwq), (dyk, ck, sk, rk, wk, dk, dwk) = args
    ws = workspace(coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, D))
    coat.coat_qk_norm_rope_ckpt_backward(dyq, dyk, cq, sq, rq, ck, sk, rk, wq, wk, cos, sin, pos, G, dq, dk, dwq, dwk, ws,
                                         interleaved=inter)
    for dy, xv, rstd, w, dx, dw in sides:
        D64 = dy.double()
        rx, rw, _, _ = R.qk_backward(D64, xv, rstd.double(), w.double(), c, s, rot, inter)
        # sizes of what is added up, the two products of a pair included
        size = R.rotate(D64.abs(), c.abs(), -s.abs(), rot, inter).abs() + R.rotate(D64.abs(), c.abs(), s.abs(), rot, inter).abs()
        _, _, sx, sw = R.rmsnorm_backward(size, xv, rstd.double(), w.double())
        near(dx, rx, bf16_bound(rx) + 2.0 ** -18 * sx, "dx")
        near(dw, rw, bf16_bound(rw) + (M * dy.shape[1] + 64) * E * sw, "dweight")
    if Hk:
        assert torch.isnan(buf[:, (Hq + Hk) * D:]).all(), "written behind the heads"


@pytest.mark.parametrize("bad", [-1, 97, 2 ** 31 - 1, -2 ** 31])
def test_a_position_outside_the_tables_shows(bad):
    M, H, D, rot, G = 4, 3, 64, 32, 16
    q, _, cos, sin, pos = qk_inputs(M, H, 0, D, rot, 3)
    pos[2] = bad
    y, codes, scale, rstd = empty(M, H, D), empty(M, H, D, dtype=U8), empty(M, H, D // G, dtype=F32), empty(M, H, dtype=F32)
    coat.coat_qk_norm_rope_ckpt(q, None, norm_w(D, 1), None, EPS, cos, sin, pos, G, y, codes, scale, rstd)
    assert torch.isnan(y[2, :, :rot]).all()
    assert torch.isfinite(y[2, :, rot:]).all() and torch.isfinite(y[[0, 1, 3]]).all()
    check_checkpoint(codes, scale, q, G, "checkpoint")


# M, N, K, G, row, col
WGRAD = [(1, 8, 16, 8, False, False), (1, 264, 272, 16, True, True), (7, 64, 128, 128, True, False), (63, 256, 256, 32, False, True),
         (64, 256, 256, 128, False, False), (65, 512, 384, 64, True, True), (1111, 520, 400, 16, False, False),
         (4096, 256, 128, 8, True, True), (300, 1376, 2048, 128, True, True), (8191, 16, 48, 16, False, True),
         (2048, 2048, 1024, 64, False, False)]


@pytest.mark.parametrize("M,N,K,G,row,col", WGRAD)
def test_weight_gradient(M, N, K, G, row, col):
    x = acts(M, K, M + K)
    q, S, xv = checkpoint(x, G)
    wide = grads(M, N + 16, M + N)
    wide[:, N:] = float("nan")                  # what lies between the rows is not read into a result
    dy = wide[:, :N]
    r = torch.rsqrt(x.float().square().mean(-1) + EPS) if row else None
    c = norm_w(K, 8) if col else None
    dw = empty(N, K)
    ws = workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K))
    coat.coat_ckpt_weight_grad(dy, q, S, G, dw, ws, row_scale=r, col_scale=c)
    torch.cuda.synchronize()
    assert coat.coat_kernel_wait_timeouts(reset=True) == 0
    ref, size = R.weight_grad(dy.double(), xv, None if r is None else r.double(), None if c is None else c.double())
    near(dw, ref, bf16_bound(ref) + (U + (M + 8) * 2.0 ** -22) * size, "dw")
    dw2 = empty(N, K)
    ws.fill_(0x7F)
    coat.coat_ckpt_weight_grad(dy, q, S, G, dw2, ws, row_scale=r, col_scale=c)
    assert torch.equal(dw, dw2), "two calls differ"


def test_weight_gradient_of_small_whole_numbers_is_exact():
    """Sums of whole numbers below 2^8 in every place: no rounding anywhere, so every index shows."""
    M, N, K, G = 40, 264, 304, 16
    dy = torch.zeros(M, N, device="cuda")
    q = torch.zeros(M, K, device="cuda")
    # column n of dy and column k of x meet in few tokens; the products name both
    for m in range(M):
        dy[m, m::M] = 1 + (torch.arange(m, N, M, device="cuda") % 13)
        q[m, m::M] = 1 + (torch.arange(m, K, M, device="cuda") % 8)
    dw = empty(N, K)
    S = torch.full((M, K // G), 0.5, device="cuda")
    codes = q.to(E4M3).view(U8)
    coat.coat_ckpt_weight_grad(dy.to(BF), codes, S, G, dw, workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K)))
    assert torch.equal(dw.double(), dy.double().T @ (q.double() / 2))


def test_checkpoints_are_the_activation_quantizers():
    M, N, G = 64, 512, 32
    x = acts(M, N, 77)
    q0, S0 = empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)
    coat.coat_act_quantize_fp8(x, G, q0, S0)
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, norm_w(N, 1), EPS, G, y, q, S, rstd)
    assert torch.equal(q, q0) and torch.equal(S, S0)
    h, uq, us = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)
    q.fill_(0xFF)
    coat.coat_swiglu_ckpt(x, x.clone(), G, h, q, S, uq, us)
    assert torch.equal(q, q0) and torch.equal(uq, q0) and torch.equal(us, S0)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -110, 2.0 ** 100])
def test_checkpoints_at_the_ends_of_the_range(scale):
    """Subnormal scales take the division; the norm of tiny rows is eps's alone, and bf16 subnormals count."""
    M, N, G = 8, 256, 8
    x = (torch.randn(M, N, generator=gen(4), device="cuda").double() * scale).to(BF)
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    if scale < 1:
        coat.coat_rmsnorm_ckpt(x, norm_w(N, 1), EPS, G, y, q, S, rstd)
        ref, rr = R.rmsnorm(x.double(), norm_w(N, 1).double(), EPS)
        near(rstd, rr, 2.0 ** -19 * rr, "rstd")
        near(y, ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), "y")
    else:                                        # squares of these overflow: only the checkpoint is asked for
        h, uq, us = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)
        coat.coat_swiglu_ckpt(x, torch.zeros_like(x), G, h, q, S, uq, us)
        assert not h.float().any() and not uq.any() and not us.any()
    check_checkpoint(q, S, x, G, "checkpoint")


def test_gate_far_from_zero():
    g = torch.tensor([-3e38, -1e4, -200.0, -100.0, -88.0, -87.0, -60.0, -20.0, 20.0, 60.0, 88.0, 100.0, 1e4, 3e38, 0.0, -0.0],
                     device="cuda").to(BF).repeat(2, 1)
    u = torch.ones_like(g)
    M, N, G = 2, 16, 8
    h, gq, uq = empty(M, N), empty(M, N, dtype=U8), empty(M, N, dtype=U8)
    gs, us = empty(M, N // G, dtype=F32), empty(M, N // G, dtype=F32)
    coat.coat_swiglu_ckpt(g, u, G, h, gq, gs, uq, us)
    ref = R.swiglu(g.double(), u.double())
    near(h, ref, bf16_bound(ref) + silu_bound(ref, g.double().abs().clamp_max(200.0)), "h")
    # backward, on values that a checkpoint holds exactly
    g = torch.tensor([-448.0, -96.0, -88.0, -24.0, 0.0, 24.0, 88.0, 448.0] * 2, device="cuda").to(BF).repeat(2, 1)
    q, S, gv = checkpoint(g, G)
    assert torch.equal(gv, g.double())
    uq, us, uv = checkpoint(u, G)
    dh = torch.ones_like(u)
    dg, du = empty(M, N), empty(M, N)
    coat.coat_swiglu_ckpt_backward(dh, q, S, uq, us, G, dg, du)
    rg, ru = R.swiglu_backward(dh.double(), gv, uv)
    s = torch.special.expit(gv)
    near(dg, rg, bf16_bound(rg) + (gv.abs() + 16) * 4 * E * (s + (gv * s).abs()) + 2.0 ** -110, "dgate")
    near(du, ru, bf16_bound(ru) + silu_bound(ru, gv) + 2.0 ** -110, "dup")


def _exact_values(M, N, G, seed):
    """Values that a checkpoint holds exactly: E4M3 values with 448 in each group, times a power of two."""
    code = torch.randint(0x20, 0x7F, (M, N), generator=gen(seed), device="cuda", dtype=torch.int32)
    code[:, ::G] = 0x7E
    sign = torch.randint(0, 2, (M, N), generator=gen(seed + 1), device="cuda", dtype=torch.int32)
    return ((code | sign << 7).to(U8).view(E4M3).double() * 2.0 ** -8).to(BF)


def test_gradients_against_differences():
    """On inputs that the checkpoint holds exactly, the backward kernels' results are the derivatives of the
    operators: central differences of the float64 forward forms, in a few random directions."""
    M, N, G = 4, 64, 16
    x, w, dy = _exact_values(M, N, G, 1), norm_w(N, 2), grads(M, N, 3)
    q, S, xv = checkpoint(x, G)
    assert torch.equal(xv, x.double())
    rstd = R.rmsnorm(xv, w.double(), EPS)[1].float()
    dx, dw = empty(M, N), empty(N)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw, workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N)))
    g, u = xv, _exact_values(M, N, G, 5)
    uq, us, uv = checkpoint(u, G)
    dg, du = empty(M, N), empty(M, N)
    coat.coat_swiglu_ckpt_backward(dy, q, S, uq, us, G, dg, du)
    cos, sin = rope_tables(97, 16)
    pos = torch.tensor([0, 5, 96, 33], device="cuda", dtype=torch.int32)
    c, s = cos[pos.long()].double(), sin[pos.long()].double()
    x3, wd, dy3 = xv.view(M, 2, 32), norm_w(32, 7), dy.view(M, 2, 32)
    r3 = R.rmsnorm(x3, wd.double(), EPS)[1].float()
    dq, dwq = empty(M, 2, 32), empty(32)
    coat.coat_qk_norm_rope_ckpt_backward(dy3, None, q.view(M, 2, 32), S.view(M, 2, 2), r3, None, None, None, wd, None, cos, sin,
                                         pos, G, dq, None, dwq, None,
                                         workspace(coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, 32)))
    D, D3 = dy.double(), dy3.double()
    cases = [(lambda t: (R.rmsnorm(t, w.double(), EPS)[0] * D).sum(), xv, dx), (lambda t: (R.rmsnorm(xv, t, EPS)[0] * D).sum(), w.double(), dw),
             (lambda t: (R.swiglu(t, uv) * D).sum(), g, dg), (lambda t: (R.swiglu(g, t) * D).sum(), uv, du),
             (lambda t: (R.qk(t, wd.double(), EPS, c, s, 16, False)[0] * D3).sum(), x3, dq),
             (lambda t: (R.qk(x3, t, EPS, c, s, 16, False)[0] * D3).sum(), wd.double(), dwq)]
    for i, (f, at, got) in enumerate(cases):
        for k in range(4):
            v = torch.randn(at.shape, generator=gen(100 + 10 * i + k), device="cuda", dtype=torch.float64)
            h = 1e-5
            diff = (f(at + h * v) - f(at - h * v)) / (2 * h)
            # each entry of the result is within u |entry| and float32's errors of the derivative
            bound = 2 * U * (got.double().abs() * v.abs()).sum() + 1e-6 * (got.double().norm() * v.norm())
            assert abs((got.double() * v).sum() - diff) <= bound, i


def test_norm_factors_let_one_checkpoint_serve_the_linear_layer():
    """dW of the layer behind a norm from the norm input's checkpoint = dW from the norm's own output, up to
    the checkpoint's grid: on inputs it holds exactly, up to bf16 rounding."""
    M, N, K, G = 96, 64, 128, 32
    x, w, dy = _exact_values(M, K, G, 9), norm_w(K, 3), grads(M, N, 4)
    y, q, S, rstd = empty(M, K), empty(M, K, dtype=U8), empty(M, K // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, rstd)
    dw = empty(N, K)
    coat.coat_ckpt_weight_grad(dy, q, S, G, dw, workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K)), row_scale=rstd, col_scale=w)
    ref = dy.double().T @ R.rmsnorm(x.double(), w.double(), EPS)[0]
    size = dy.double().abs().T @ R.rmsnorm(x.double(), w.double(), EPS)[0].abs()
    near(dw, ref, bf16_bound(ref) + (U + 2.0 ** -14) * size, "dw")


def test_another_stream_and_a_graph():
    """The calls run on the stream that they are given, and record into a graph."""
    M, N, G = 130, 1024, 64
    x, w = acts(M, N, 5), norm_w(N, 6)
    y0, q0, S0, r0 = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y0, q0, S0, r0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, q, S, r = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    dx, dw = empty(M, N), empty(N)
    dwl = empty(256, N)
    dy, dyl = grads(M, N, 7), grads(M, 256, 8)
    ws = workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N))
    ws2 = workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, 256, N))
    late = torch.zeros_like(x)

    def step(stream=None):
        coat.coat_rmsnorm_ckpt(late, w, EPS, G, y, q, S, r, stream=stream)
        coat.coat_rmsnorm_ckpt_backward(dy, q, S, r, w, G, dx, dw, ws, stream=stream)
        coat.coat_ckpt_weight_grad(dyl, q, S, G, dwl, ws2, stream=stream)

    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    step(stream=side)                            # named: the current stream is another one
    side.synchronize()
    assert torch.equal(y, y0) and torch.equal(q, q0) and torch.equal(S, S0) and torch.equal(r, r0)
    dx0, dw0, dwl0 = dx.clone(), dw.clone(), dwl.clone()
    for t in (y, dx, dw, dwl):
        t.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dw, dw0) and torch.equal(dwl, dwl0)


def test_the_binding_refuses_wrong_tensors():
    M, N, G = 16, 64, 16
    x, w = acts(M, N, 1), norm_w(N, 1)
    y, q, S, r = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    with pytest.raises(TypeError):
        coat.coat_rmsnorm_ckpt(x.float(), w, EPS, G, y, q, S, r)
    with pytest.raises(TypeError):
        coat.coat_rmsnorm_ckpt(x, w.to(BF), EPS, G, y, q, S, r)
    with pytest.raises(ValueError):
        coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S[:-1], r)
    with pytest.raises(ValueError):
        coat.coat_rmsnorm_ckpt(x[:, ::2], w[:32], EPS, G, y, q, S, r)
    with pytest.raises(ValueError):
        coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, r, residual=x.clone())
    with pytest.raises(ValueError):
        coat.coat_rmsnorm_ckpt(x.cpu(), w, EPS, G, y, q, S, r)
    with pytest.raises(coat.CoatError) as e:
        coat.coat_rmsnorm_ckpt(x, w, 0.0, G, y, q, S, r)
    assert e.value.status == 1
    with pytest.raises(coat.CoatError) as e:
        coat.coat_rmsnorm_ckpt(x, w, EPS, G, x, q, S, r)
    assert e.value.status == 1
    with pytest.raises(coat.CoatError) as e:             # a workspace that is too small
        coat.coat_rmsnorm_ckpt_backward(x, q, S, r, w, G, y, empty(N), workspace(16))
    assert e.value.status == 1
    with pytest.raises(ValueError):                      # a row's elements apart
        coat.coat_swiglu_ckpt(acts(M, 2 * N, 1)[:, ::2], x, G, y, q, S, q.clone(), S.clone())
    with pytest.raises(ValueError):                      # strides that differ
        coat.coat_swiglu_ckpt(acts(M, 2 * N, 1)[:, :N], x, G, y, q, S, q.clone(), S.clone())
    with pytest.raises(ValueError):
        coat.coat_ckpt_weight_grad(x, q[0], S, G, empty(N, N), workspace(16))
    with pytest.raises(coat.CoatError) as e:
        coat.coat_ckpt_weight_grad(x, q, empty(M, N // 4, dtype=F32), 4, empty(N, N), workspace(16))
    assert e.value.status == 3
    assert math.isfinite(w.sum().item())                 # nothing left the device in error
