"""The operators as a step uses them: lookup, dropout into the residual stream, the norm with its 8-bit checkpoint, the cross
entropy, all gradients back into one flat bf16 gradient of a tied table, and the optimizer's step, all in one captured graph
that is replayed on other data, against the same calls made one by one."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, F32, U8, embedding, embedding_backward, gen, linear_cross_entropy, linear_cross_entropy_backward, randn

pytestmark = pytest.mark.gpu
M, V, C, G, EPS, P = 300, 1111, 256, 32, 1e-5, 0.2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    coat.lib()


class Step:
    """A table, one norm, the tied output layer; every tensor kept, so that the calls can be captured."""

    def __init__(self):
        n = V * C + C
        self.flat, self.grad = randn(n, seed=1) * 0.05, torch.empty(n, dtype=BF, device="cuda")
        self.flat[V * C:] = 1.0
        self.flat16 = self.flat.to(BF)
        self.table, self.dtable, self.dnorm = self.flat16[:V * C].view(V, C), self.grad[:V * C].view(V, C), self.grad[V * C:]
        self.m_q, self.v_q = torch.zeros(n, dtype=U8, device="cuda"), torch.zeros(n, dtype=U8, device="cuda")
        self.meta = torch.tensor([0.0, 1.0, 0.0, 1.0], device="cuda").repeat(coat.num_groups(n, 128), 1)
        self.ids, self.targets = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(2))
        self.rng, self.res = torch.tensor([5, 0], device="cuda"), torch.empty(M, C, dtype=BF, device="cuda")
        self.x, self.d, self.y, self.dy, self.dx, self.dd, self.h = (torch.empty(M, C, dtype=BF, device="cuda") for _ in range(7))
        self.q, self.scale = torch.empty(M, C, dtype=U8, device="cuda"), torch.empty(M, C // G, device="cuda")
        self.rstd, self.loss, self.lse = (torch.empty(M, device="cuda") for _ in range(3))
        self.dloss = torch.empty(M, device="cuda")
        self.ws = torch.empty(max(coat.coat_rmsnorm_ckpt_backward_workspace_bytes(M, C),
                                  coat.coat_linear_cross_entropy_workspace_bytes(M, V),
                                  coat.coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, 512),
                                  coat.coat_embedding_backward_workspace_bytes(M, V, C)), dtype=U8, device="cuda")

    def data(self, seed):
        self.ids.copy_(torch.randint(-1, V, (M,), generator=gen(seed), device="cuda"))
        t = torch.randint(0, V, (M,), generator=gen(seed + 1), device="cuda")
        t[::9] = -100
        self.targets.copy_(t)
        self.dloss.copy_((t >= 0).float() / (t >= 0).sum())
        self.res.copy_(randn(M, C, seed=seed + 2))

    def calls(self):
        norm = self.flat[V * C:]
        coat.coat_embedding(self.table, self.ids, 4.0, self.x)
        coat.coat_dropout(self.x, P, self.rng, self.d)
        coat.coat_rmsnorm_ckpt(self.d, norm, EPS, G, self.y, self.q, self.scale, self.rstd, residual=self.res, h=self.h)
        coat.coat_linear_cross_entropy(self.y, self.table, self.targets, self.loss, self.lse, self.ws)
        coat.coat_linear_cross_entropy_backward(self.y, self.table, self.targets, self.lse, self.dloss, self.dy, self.dtable, self.ws,
                                                piece=512)
        coat.coat_rmsnorm_ckpt_backward(self.dy, self.q, self.scale, self.rstd, norm, G, self.dx, self.dnorm, self.ws)
        coat.coat_dropout_backward(self.dx, P, self.rng, self.dd)
        coat.coat_embedding_backward(self.dd, self.ids, 4.0, self.dtable, self.ws, accumulate=True)
        coat.coat_fp8_adamw_step(self.flat, self.grad, self.m_q, self.v_q, self.meta, 128, 0.9, 0.95, 1e-3, 1e-8, 0.1, 1)
        self.rng[1] += 1

    def state(self):
        return [t.clone() for t in (self.loss, self.lse, self.grad, self.flat, self.m_q, self.v_q, self.meta, self.rng)]


def test_captured_and_replayed():
    a, b = Step(), Step()
    a.data(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = [(t, t.clone()) for t in (a.flat, a.m_q, a.v_q, a.meta, a.rng)]
    with torch.cuda.stream(s):
        a.calls()
    s.synchronize()
    for t, old in saved:
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.calls()
    for seed in (10, 20, 30):
        a.data(seed)
        b.data(seed)
        graph.replay()
        b.calls()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x.view(U8), y.view(U8))
        a.flat16.copy_(a.flat)
        b.flat16.copy_(b.flat)


def test_the_tied_gradient_is_the_sum_of_both_ends():
    """Each end against float64 of what went into it; the sum is rounded to bf16 at the first end and once more at the second."""
    a = Step()
    a.data(3)
    a.calls()
    _, rlse, _, _ = linear_cross_entropy(a.y, a.table, a.targets)
    assert ((a.lse.double() - rlse).abs() <= 1e-5 * rlse.abs().clamp_min(1)).all()
    _, head, _, size, _, _, _ = linear_cross_entropy_backward(a.y, a.table, a.targets, a.lse, a.dloss)
    low, terms, _ = embedding_backward(a.dd, a.ids, 4.0, V)
    want = head + low
    bound = 2.0 ** -7 * (size + head.abs()) + 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -16 * terms + 2.0 ** -100
    assert ((a.dtable.double() - want).abs() <= bound).all()
    ref = embedding(a.table, a.ids, 4.0)
    assert ((a.x.double() - ref).abs() <= 2.0 ** -8 * ref.abs()).all()
    assert a.loss.dtype == F32


def several(tokens):
    """Both directions of the cross entropy and of the embedding, with a workspace of their own; their results."""
    m, v, c = tokens, 2500, 192
    x, w = randn(m, c, seed=tokens).to(BF), (randn(v, c, seed=tokens + 1) * 0.1).to(BF)
    t = torch.randint(-1, v, (m,), generator=gen(tokens + 2), device="cuda")
    g = torch.rand(m, generator=gen(tokens + 3), device="cuda")
    ws = torch.empty(max(coat.coat_linear_cross_entropy_workspace_bytes(m, v),
                         coat.coat_linear_cross_entropy_backward_workspace_bytes(m, v, c, 1024),
                         coat.coat_embedding_backward_workspace_bytes(m, v, c)), dtype=U8, device="cuda")
    out = [torch.zeros(s, dtype=d, device="cuda") for s, d in (((m,), F32), ((m,), F32), ((m, c), BF), ((v, c), BF), ((v, c), BF), ((m, c), BF))]

    def calls(stream=None):
        loss, lse, dx, dw, dtable, rows = out
        coat.coat_linear_cross_entropy(x, w, t, loss, lse, ws, stream=stream)
        coat.coat_linear_cross_entropy_backward(x, w, t, lse, g, dx, dw, ws, piece=1024, stream=stream)
        coat.coat_embedding_backward(dx, t, 1.5, dtable, ws, stream=stream)
        coat.coat_embedding(w, t, 2.0, rows, stream=stream)
    return calls, out


@pytest.mark.parametrize("threads", [False, True])
def test_calls_on_several_streams_at_once(threads):
    """As one by one, bit for bit, whichever streams they are on and whichever threads make the calls."""
    import threading
    work = [several(n) for n in (40, 700, 1500)]
    want = []
    for calls, out in work:
        calls()
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
        for o in out:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    if threads:
        def run(k):
            for _ in range(20):
                work[k][0](streams[k])
        every = [threading.Thread(target=run, args=(k,)) for k in range(len(work))]
        for th in every:
            th.start()
        for th in every:
            th.join()
    else:
        for _ in range(20):
            for (calls, _), s in zip(work, streams):
                calls(s)
    torch.cuda.synchronize()
    for (_, out), ref in zip(work, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert coat.coat_kernel_wait_timeouts(reset=True) == 0


@pytest.mark.parametrize("which", ["cross entropy", "its gradients", "linear", "weight gradient"])
def test_the_first_call_of_a_thread(which):
    """A thread that has done nothing on the device before has no current CUDA context; the calls that lay out
    copies by it take the device's."""
    import threading
    m, n, k = 256, 256, 256
    g = gen(3)
    xq, wq = (torch.randint(0, 100, (s, k), generator=g, device="cuda").to(U8) for s in (m, n))
    x, w, dy = randn(m, k, seed=1).to(BF), randn(n, k, seed=2).to(BF), randn(m, n, seed=3).to(BF)
    t, one = torch.arange(m, device="cuda") % n, torch.ones(m, device="cuda")
    lse = linear_cross_entropy(x, w, t)[1].float()
    scale = torch.ones(m, k // 128, device="cuda")
    ws = torch.empty(1 << 24, dtype=U8, device="cuda")

    def call(a, b):
        if which == "cross entropy":
            coat.coat_linear_cross_entropy(x, w, t, a[:m], b[:m], ws)
        elif which == "its gradients":
            coat.coat_linear_cross_entropy_backward(x, w, t, lse, one, a.view(BF)[:m * k].view(m, k), b.view(BF)[:n * k].view(n, k), ws)
        elif which == "linear":
            coat.coat_fp8_linear_group_quantize(xq, 1.0, wq, 1.0, 128, a.view(U8)[:m * n].view(m, n), b[:m * n // 128].view(m, n // 128))
        else:
            coat.coat_ckpt_weight_grad(dy, xq, scale, 128, a.view(BF)[:n * k].view(n, k), ws)
    out = [torch.zeros(m * k, device="cuda") for _ in range(4)]
    wrong = []

    def run():
        try:
            call(*out[:2])
        except Exception as e:   # a thread's exceptions do not reach the test by themselves
            wrong.append(e)
    torch.cuda.synchronize()
    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    assert not wrong, wrong
    call(*out[2:])
    torch.cuda.synchronize()
    assert out[0].any() and torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
