"""The operators with 8-bit activation checkpoints where they can go wrong: every
bf16 quotient, many widths, pointers and strides that only the documented
alignment holds for, offsets past 32 bits, and the weight gradient's split
tiles.  Forms and bounds as in test_gpu_ckpt.py."""
import pytest
import torch

import _ckpt_ref as R
import coat_fp8_adamw_gb300 as coat
from test_gpu_ckpt import (BF, E, E4M3, EPS, F32, U, U8, acts, bf16_bound, check_checkpoint, checkpoint, empty, gen, grads,
                           near, norm_w, rope_tables, silu_bound, workspace)
from test_gpu_ckpt import _built  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu


def _all_quotients():
    """Groups of eight: a largest value of every bf16 significand and seven more, so that every pair of significands
    meets at every distance of the exponents that a code other than zero can have, and beyond."""
    sig = 1 + torch.arange(128, dtype=torch.float64) / 128
    x = (sig[:, None] * torch.exp2(-torch.arange(21, dtype=torch.float64))).flatten()       # 2688 = 7 * 384
    x = x * torch.where(torch.arange(x.numel()) % 3 == 0, -1.0, 1.0)
    groups = torch.empty(128, x.numel() // 7, 8, dtype=torch.float64)
    groups[:, :, 0] = 2 * sig[:, None]
    groups[:, :, 1:] = x.view(-1, 7)
    return groups.view(-1, 128)                                                             # 16 groups a row


@pytest.mark.parametrize("power", [0, -40, 90, -90, -104, 124])
def test_every_bf16_quotient_is_rounded_like_the_exact_one(power):
    x = (_all_quotients() * 2.0 ** power).cuda().to(BF)       # the lowest of 2^-104 .. 2^-126 stay normal
    M, N = x.shape
    G = 8
    h, gq, uq = empty(M, N), empty(M, N, dtype=U8), empty(M, N, dtype=U8)
    gs, us = empty(M, N // G, dtype=F32), empty(M, N // G, dtype=F32)
    coat.coat_swiglu_ckpt(x, -x, G, h, gq, gs, uq, us)
    check_checkpoint(gq, gs, x, G, "gate")
    check_checkpoint(uq, us, -x, G, "up")
    if power > 0:
        return                                                # squares overflow: no norm of these
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, norm_w(N, 1), EPS, G, y, q, S, rstd)
    assert torch.equal(q, gq) and torch.equal(S, gs)
    q.fill_(0xFF)
    cos, sin = rope_tables(4, 32)
    coat.coat_qk_norm_rope_ckpt(x.view(M, 2, 64), None, norm_w(64, 1), None, EPS, cos, sin,
                                torch.zeros(M, dtype=torch.int32, device="cuda"), G, y.view(M, 2, 64), q.view(M, 2, 64),
                                S.view(M, 2, 8), empty(M, 2, dtype=F32))
    assert torch.equal(q, gq) and torch.equal(S, gs)


def _norm_both_ways(M, N, G, seed, res):
    x, w, dy = acts(M, N, seed), norm_w(N, seed), grads(M, N, seed + 3)
    dres = grads(M, N, seed + 4) if res else None
    h = empty(M, N) if res else None
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, rstd, residual=torch.zeros_like(x) if res else None, h=h)
    ref, rr = R.rmsnorm(x.double(), w.double(), EPS)
    what = f"{M}x{N} G={G} "
    near(rstd, rr, 2.0 ** -19 * rr, what + "rstd")
    near(y, ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), what + "y")
    check_checkpoint(q, S, x, G, what)
    xv = R.dequantize(q.view(E4M3).double(), S.double(), G)
    dx, dw = empty(M, N), empty(N)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw,
                                    workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N)), dresidual=dres)
    rx, rw, sx, sw = R.rmsnorm_backward(dy.double(), xv, rstd.double(), w.double())
    rx = rx if dres is None else rx + dres.double()
    near(dx, rx, bf16_bound(rx) + 2.0 ** -18 * sx + 2 * E * rx.abs(), what + "dx")
    near(dw, rw, bf16_bound(rw) + (M + 64) * E * sw, what + "dweight")


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("res", [False, True])
def test_norm_of_many_widths(G, res):
    for N in (*range(16, 2100, 112), 2560, 4080, 4096, 4112, 4912, 4928, 6144, 8176, 8208, 12288, 16384):
        _norm_both_ways(37, N, G, N, res)


@pytest.mark.parametrize("M", [151, 152, 153, 607, 1217, 5000])
def test_norm_of_many_rows(M):
    for N, G in ((64, 64), (1008, 16), (4096, 128)):
        _norm_both_ways(M, N, G, M + N, True)


def _off(t, n):
    """t's values in memory that starts n elements behind a 256-byte boundary."""
    b = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
    b[n:] = t.flatten()
    return b[n:].view(t.shape)


@pytest.mark.parametrize("N,G", [(48, 16), (528, 8), (1024, 128), (4112, 16)])
def test_pointers_on_sixteen_bytes_only(N, G):
    M = 19
    x, w, dy = acts(M, N, 3), norm_w(N, 4), grads(M, N, 5)
    want = [empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)]
    got = [_off(t, 16 // t.element_size()) for t in want]
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, *want)
    coat.coat_rmsnorm_ckpt(_off(x, 8), _off(w, 4), EPS, G, *got)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    _, q, S, rstd = want
    bytes_ = coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N)
    dx, dw, dx2, dw2 = empty(M, N), empty(N), _off(empty(M, N), 8), _off(empty(N), 8)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw, workspace(bytes_))
    coat.coat_rmsnorm_ckpt_backward(_off(dy, 8), *got[1:], _off(w, 4), G, dx2, dw2, _off(workspace(bytes_), 16))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)

    ins = [acts(M, N, 6), acts(M, N, 7)]
    want = [empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)]
    got = [_off(t, 16 // t.element_size()) for t in want]
    coat.coat_swiglu_ckpt(*ins, G, *want)
    coat.coat_swiglu_ckpt(*[_off(t, 8) for t in ins], G, *got)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = [empty(M, N), empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)]
    out2 = [_off(t, 16 // t.element_size()) for t in out]
    coat.coat_swiglu_ckpt_backward(dy, *want[1:], G, *out[:2], h_q=out[2], h_scale=out[3])
    coat.coat_swiglu_ckpt_backward(_off(dy, 8), *got[1:], G, *out2[:2], h_q=out2[2], h_scale=out2[3])
    assert all(torch.equal(a, b) for a, b in zip(out, out2))

    K = N
    dyw = grads(M, 136, 8)
    dw, dw2 = empty(136, K), _off(empty(136, K), 8)
    bytes_ = coat.coat_ckpt_weight_grad_workspace_bytes(M, 136, K)
    r = torch.rand(M, device="cuda")
    coat.coat_ckpt_weight_grad(dyw, want[1], want[2], G, dw, workspace(bytes_), row_scale=r, col_scale=w)
    coat.coat_ckpt_weight_grad(_off(dyw, 8), got[1], got[2], G, dw2, _off(workspace(bytes_), 16), row_scale=_off(r, 4),
                               col_scale=_off(w, 4))
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("D,rot,G,inter", [(48, 32, 16, False), (128, 128, 128, True), (80, 64, 8, False)])
def test_heads_on_sixteen_bytes_only(D, rot, G, inter):
    M, Hq, Hk = 21, 6, 2
    wide = acts(M, (Hq + 2 * Hk) * D + 8, 2)
    cos, sin = rope_tables(50, rot)
    pos = torch.randint(0, 50, (M,), generator=gen(1), device="cuda", dtype=torch.int32)
    q, k = wide[:, 8:8 + Hq * D].view(M, Hq, D), wide[:, 8 + Hq * D:8 + (Hq + Hk) * D].view(M, Hk, D)
    w = [norm_w(D, 1), norm_w(D, 2)]
    runs, grads_ = [], []
    dy = [grads(M, H * D, 9).view(M, H, D) for H in (Hq, Hk)]
    for n in (0, 1):
        o = [[_off(empty(M, H, D), 8 * n), _off(empty(M, H, D, dtype=U8), 16 * n), _off(empty(M, H, D // G, dtype=F32), 4 * n),
              _off(empty(M, H, dtype=F32), 4 * n)] for H in (Hq, Hk)]
        a, b = (q, k) if n else (q.contiguous(), k.contiguous())
        args = [_off(t, 4 * n) for t in (*w, cos, sin, pos)]
        coat.coat_qk_norm_rope_ckpt(a, b, args[0], args[1], EPS, *args[2:], G, *o[0], *o[1], interleaved=inter)
        runs.append(o[0] + o[1])
        dq, dk = (_off(empty(M, H, D), 8 * n) for H in (Hq, Hk))
        dwq, dwk = _off(empty(D), 8 * n), _off(empty(D), 8 * n)
        coat.coat_qk_norm_rope_ckpt_backward(
            _off(dy[0], 8 * n), _off(dy[1], 8 * n), *o[0][1:], *o[1][1:], *args, G, dq, dk, dwq, dwk,
            _off(workspace(coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, D)), 16 * n), interleaved=inter)
        grads_.append([dq, dwq, dk, dwk])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert all(torch.equal(a, b) for a, b in zip(*grads_))


def test_rows_past_two_to_the_32():
    """Rows 2^27 elements apart: the last ones lie behind the 2^32nd element."""
    M, N, G, ld = 36, 272, 16, 1 << 27
    big = torch.empty(M * ld, dtype=BF, device="cuda").view(M, ld)
    src = acts(M, 2 * N, 11)
    big[:, 8:8 + 2 * N] = src
    g, u = big[:, 8:8 + N], big[:, 8 + N:8 + 2 * N]
    h, gq, uq = empty(M, N), empty(M, N, dtype=U8), empty(M, N, dtype=U8)
    gs, us = empty(M, N // G, dtype=F32), empty(M, N // G, dtype=F32)
    coat.coat_swiglu_ckpt(g, u, G, h, gq, gs, uq, us)
    check_checkpoint(gq, gs, src[:, :N], G, "gate")
    check_checkpoint(uq, us, src[:, N:], G, "up")
    dh = grads(M, N, 12)
    want = [empty(M, N), empty(M, N)]
    coat.coat_swiglu_ckpt_backward(dh, gq, gs, uq, us, G, *want)
    coat.coat_swiglu_ckpt_backward(dh, gq, gs, uq, us, G, g, u)
    assert torch.equal(g, want[0]) and torch.equal(u, want[1])

    D, rot, H = 16, 16, 17
    big[:, 8:8 + 2 * N] = src
    q, k = big[:, 8:8 + N].view(M, H, D), big[:, 8 + N:8 + 2 * N].view(M, H, D)
    cos, sin = rope_tables(M, rot)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    w = norm_w(D, 3)
    outs = []
    for a, b in ((q, k), (q.contiguous(), k.contiguous())):
        o = [[empty(M, H, D), empty(M, H, D, dtype=U8), empty(M, H, 1, dtype=F32), empty(M, H, dtype=F32)] for _ in "qk"]
        coat.coat_qk_norm_rope_ckpt(a, b, w, w, EPS, cos, sin, pos, D, *o[0], *o[1])
        outs.append(o[0] + o[1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    o, dy = outs[0], grads(M, N, 13).view(M, H, D)
    ws = workspace(coat.coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, D))
    res = []
    for dq, dk in ((empty(M, H, D), empty(M, H, D)), (q, k)):
        dwq, dwk = empty(D), empty(D)
        coat.coat_qk_norm_rope_ckpt_backward(dy, dy, *o[1:4], *o[5:8], w, w, cos, sin, pos, D, dq, dk, dwq, dwk, ws)
        res.append([dq, dk, dwq, dwk])
    assert all(torch.equal(a, b) for a, b in zip(*res))

    big[:, 8:8 + N] = dh
    a, b = empty(N, N), empty(N, N)
    ws = workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, N))
    coat.coat_ckpt_weight_grad(big[:, 8:8 + N], gq, gs, G, a, ws)
    coat.coat_ckpt_weight_grad(dh, gq, gs, G, b, ws)
    assert torch.equal(a, b)


def test_norm_with_more_than_two_to_the_31_elements():
    M, N, G = (1 << 17) + 5, 16384, 128
    rows = [0, 1, (1 << 16) - 1, 1 << 16, (1 << 17) - 1, 1 << 17, M - 1]
    some, w = acts(len(rows), N, 21), norm_w(N, 22)
    x = torch.zeros(M, N, dtype=BF, device="cuda")
    x[rows] = some
    y, q = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, N, dtype=U8, device="cuda")
    S, rstd = torch.empty(M, N // G, device="cuda"), torch.empty(M, device="cuda")
    coat.coat_rmsnorm_ckpt(x, w, EPS, G, y, q, S, rstd)
    ref, rr = R.rmsnorm(some.double(), w.double(), EPS)
    near(y[rows], ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), "y")
    check_checkpoint(q[rows], S[rows], some, G, "checkpoint")
    assert int(y.view(torch.int16).ne(0).any(1).sum()) <= len(rows)
    dy = x.zero_()
    dy[rows] = g = grads(len(rows), N, 23)
    dx, dw = y, empty(N)
    coat.coat_rmsnorm_ckpt_backward(dy, q, S, rstd, w, G, dx, dw,
                                    workspace(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N)))
    xv = R.dequantize(q[rows].view(E4M3).double(), S[rows].double(), G)
    rx, rw, sx, sw = R.rmsnorm_backward(g.double(), xv, rstd[rows].double(), w.double())
    near(dx[rows], rx, bf16_bound(rx) + 2.0 ** -18 * sx + 2 * E * rx.abs(), "dx")
    near(dw, rw, bf16_bound(rw) + (len(rows) + 64) * E * sw, "dweight")


def test_weight_gradient_of_a_million_tokens():
    """dY and the codes have more than 2^31 elements; tokens of both ends and of the middle count."""
    M, N, K, G = (1 << 20) + 77, 2056, 2064, 16
    rows = torch.tensor([0, 5, 63, 64, 1 << 19, (1 << 20) - 1, 1 << 20, M - 70, M - 2, M - 1], device="cuda")
    x, g = acts(len(rows), K, 31), grads(len(rows), N, 32)
    q, S, xv = checkpoint(x, G)
    dy = torch.zeros(M, N, dtype=BF, device="cuda")
    codes = torch.full((M, K), 0x38, dtype=U8, device="cuda")
    scale = torch.ones(M, K // G, device="cuda")
    dy[rows], codes[rows], scale[rows] = g, q, S
    dw = empty(N, K)
    coat.coat_ckpt_weight_grad(dy, codes, scale, G, dw, workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    assert coat.coat_kernel_wait_timeouts(reset=True) == 0
    ref, size = R.weight_grad(g.double(), xv)
    near(dw, ref, bf16_bound(ref) + (U + (len(rows) + 8) * 2.0 ** -22) * size, "dw")


# tiles of 256 x 256 below, at and above one and two rounds of 76 pairs, and tokens around the shortest parts
@pytest.mark.parametrize("N,K", [(256, 256), (1280, 3840), (1016, 4864), (2048, 2560), (2560, 3840), (304, 272)])
@pytest.mark.parametrize("M", [511, 512, 1023, 1025, 1600])
def test_weight_gradient_of_split_tiles(M, N, K):
    G = 8 if K == 272 else 128
    x, dy = acts(M, K, M + K), grads(M, N, N)
    q, S, xv = checkpoint(x, G)
    dw = empty(N, K)
    ws = workspace(coat.coat_ckpt_weight_grad_workspace_bytes(M, N, K))
    coat.coat_ckpt_weight_grad(dy, q, S, G, dw, ws)
    torch.cuda.synchronize()
    assert coat.coat_kernel_wait_timeouts(reset=True) == 0
    ref, size = R.weight_grad(dy.double(), xv)
    near(dw, ref, bf16_bound(ref) + (U + (M + 8) * 2.0 ** -22) * size, "dw")


@pytest.mark.parametrize("N,G", [(16, 16), (64, 8), (4096, 128)])
def test_swiglu_of_many_row_counts(N, G):
    for M in (1, 2, 5, 31, 151, 153, 1300):
        x = acts(M, 2 * N, M + N)
        g, u = x[:, :N], x[:, N:]
        h, gq, uq = empty(M, N), empty(M, N, dtype=U8), empty(M, N, dtype=U8)
        gs, us = empty(M, N // G, dtype=F32), empty(M, N // G, dtype=F32)
        coat.coat_swiglu_ckpt(g, u, G, h, gq, gs, uq, us)
        ref = R.swiglu(g.double(), u.double())
        near(h, ref, bf16_bound(ref) + silu_bound(ref, g.double()) + 2.0 ** -120 * (g.double() * u.double()).abs(), "h")
        check_checkpoint(gq, gs, g.contiguous(), G, "gate")
        check_checkpoint(uq, us, u.contiguous(), G, "up")


def test_calls_that_follow_one_another_at_once():
    """Kernels start before the one ahead of them has ended: each has to see its results, and must not write what it still
    reads.  A chain over two buffers, also behind copies, in a graph, and behind another stream's work."""
    M, N, G, D = 1031, 2048, 32, 64
    x0, w, w2 = acts(M, N, 51), norm_w(N, 52), norm_w(D, 53)
    cos, sin = rope_tables(M, D)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    a, b, c, dw, dw2 = empty(M, N), empty(M, N), empty(M, N), empty(N), empty(N // 8, N)
    q, S, rstd, rh = empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32), empty(M, N // D, dtype=F32)
    q2, S2, q3, S3 = empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32)
    ws = workspace(max(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, N),
                       coat.coat_ckpt_weight_grad_workspace_bytes(M, N // 8, N)))
    dy = grads(M, N // 8, 54)
    heads = lambda t, n=D: t.view(M, N // D, n)  # noqa: E731
    sums = torch.zeros(1, dtype=torch.float64, device="cuda")

    def chain(rounds, sync):
        for i in range(rounds):
            coat.coat_rmsnorm_ckpt(a, w, EPS, G, b, q, S, rstd)
            sync()
            coat.coat_qk_norm_rope_ckpt(heads(b), None, w2, None, EPS, cos, sin, pos, G, heads(a), heads(q), heads(S, D // G), rh)
            sync()
            coat.coat_swiglu_ckpt(a, b, G, c, q, S, q2, S2)
            sync()
            coat.coat_ckpt_weight_grad(dy, q, S, G, dw2, ws)
            sync()
            coat.coat_rmsnorm_ckpt_backward(c, q2, S2, rstd, w, G, a, dw, ws)
            sync()
            coat.coat_swiglu_ckpt_backward(a, q, S, q2, S2, G, b, c, h_q=q3, h_scale=S3)
            sync()
            coat.coat_rmsnorm_ckpt(b, w, EPS, G, a, q, S, rstd, residual=x0, h=c)
            sync()
        return [t.clone() for t in (a, b, c, dw, dw2, q, S, q2, S2, q3, S3, rstd)]

    a.copy_(x0)
    want = chain(4, torch.cuda.synchronize)
    assert all(torch.isfinite(t.double()).all() for t in want)
    for _ in range(5):
        a.zero_()
        torch.cuda.synchronize()
        a.copy_(x0)
        got = chain(4, lambda: None)
        assert all(torch.equal(u, v) for u, v in zip(want, got))

    host = x0.cpu().pin_memory()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        a.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            a.copy_(host, non_blocking=True)
        main.wait_stream(side)
        got = chain(4, lambda: None)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            sums[0] = got[0].double().sum()
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    assert sums[0] == want[0].double().sum()

    other = torch.cuda.Stream()
    a.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(2_000_000)
        a.copy_(x0)
    torch.cuda.current_stream().wait_stream(other)
    got = chain(4, lambda: None)
    assert all(torch.equal(u, v) for u, v in zip(want, got))


@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -126, 1e-12, 1.0, 3e38])
def test_every_positive_eps(eps):
    """A zero row's 1/rms is 1/sqrt(eps), also of a subnormal one; its outputs are zeros.  (The sum's last bit is 2^-149.)"""
    eps = float(torch.tensor(eps, dtype=F32))
    M, N, G, D = 5, 256, 16, 64
    x, w = acts(M, N, 61, spread=0.5), norm_w(N, 62)
    y, q, S, rstd = empty(M, N), empty(M, N, dtype=U8), empty(M, N // G, dtype=F32), empty(M, dtype=F32)
    coat.coat_rmsnorm_ckpt(x, w, eps, G, y, q, S, rstd)
    ref, rr = R.rmsnorm(x.double(), w.double(), eps)
    near(rstd, rr, 2.0 ** -19 * rr, "rstd")
    near(y, ref, bf16_bound(ref) + 2.0 ** -19 * ref.abs(), "y")
    assert not y[1].float().any()
    cos, sin = rope_tables(M, D)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    y = empty(M, N // D, D)
    rh = torch.empty(M, N // D, device="cuda")
    coat.coat_qk_norm_rope_ckpt(x.view(M, N // D, D), None, w[:D].clone(), None, eps, cos, sin, pos, G, y, q.view(M, N // D, D),
                                S.view(M, N // D, D // G), rh)
    rr = R.rmsnorm(x.double().view(M, N // D, D), w[:D].double(), eps)[1]
    near(rh, rr, 2.0 ** -19 * rr, "head rstd")
    assert not y[1].float().any()


@pytest.mark.parametrize("N", [3584, 4608, 5120, 5136, 6656, 8192, 8208, 9728, 16384])
@pytest.mark.parametrize("res", [False, True])
def test_norm_around_the_widths_where_blocks_change(N, res):
    """Rows for several rounds of one, two or three blocks per SM."""
    _norm_both_ways(1201, N, 16, N + 1, res)
