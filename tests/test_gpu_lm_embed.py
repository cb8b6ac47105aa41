"""Embedding lookup and its gradient on the GPU, through the binding, against float64.

Bounds, per element (U = 2^-8, half a bf16 step relatively; E = 2^-24): the lookup is one float32 product, rounded to bf16:
U (1 + U) |ref| + E |ref|.  The gradient adds n float32 terms in some order, (n + 2) E sum|terms| with the product by the
scale and, where it is added, the addition, and is rounded to bf16 once."""
import pytest
import torch

import coat_fp8_adamw_gb300 as coat
from _lm_ref import BF, E, U8, bf16_bound, embedding, embedding_backward, gen, near, randn, unwritten, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from coat_fp8_adamw_gb300 import _build
    _build.build()
    coat.lib()


def text(M, V, seed):
    """Ids as text has them, with some padding."""
    u = torch.rand(M, generator=gen(seed), device="cuda")
    ids = (torch.exp(u * torch.log(torch.tensor(V + 1.0))).long() - 1).clamp(0, V - 1)
    ids[torch.rand(M, generator=gen(seed + 1), device="cuda") < 0.05] = -1
    return ids


def backward(dout, ids, scale, V, old=None, ws=None, stream=None):
    M, C = dout.shape
    d = unwritten(V, C) if old is None else old.clone()
    ws = workspace(coat.coat_embedding_backward_workspace_bytes(M, V, C)) if ws is None else ws
    coat.coat_embedding_backward(dout, ids, scale, d, ws, accumulate=old is not None, stream=stream)
    return d


def check_backward(dout, ids, scale, V, old=None, what="dtable"):
    got = backward(dout, ids, scale, V, old)
    ref, size, n = embedding_backward(dout, ids, scale, V)
    if old is not None:
        assert torch.equal(got[n == 0].view(torch.int16), old[n == 0].view(torch.int16)), f"{what}: a row without a token"
        ref, size = ref + old.double(), size + old.double().abs()
    else:
        assert not got[n == 0].view(torch.int16).any(), f"{what}: a row without a token"
    bound = (n + 2).double()[:, None] * E * size + bf16_bound(ref)
    near(got[n > 0], ref[n > 0], (bound * (1 + 2.0 ** -7))[n > 0], what) if (n > 0).any() else None
    return got


SIZES = [(1, 1, 16), (1, 300, 16), (2, 7, 48), (17, 50, 2048), (31, 5, 64), (33, 1000, 528), (1000, 153, 512), (4099, 32000, 128),
         (700, 64, 5120), (257, 200003, 16), (8192, 512, 1024)]


@pytest.mark.parametrize("M,V,C", SIZES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_lookup(M, V, C, index):
    table, ids = randn(V, C, seed=M).to(BF), text(M, V, V).to(index)
    for scale in (1.0, C ** 0.5, -0.3):
        out = unwritten(M, C)
        coat.coat_embedding(table, ids, scale, out)
        ref = embedding(table, ids, torch.tensor(scale).float().double().item())
        near(out, ref, bf16_bound(ref) + 2 * E * ref.abs(), "out")
        assert not out[ids < 0].view(torch.int16).any()
        if scale == 1.0:
            assert torch.equal(out[ids >= 0], table[ids[ids >= 0].long()])


@pytest.mark.parametrize("M,V,C", SIZES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("add", [False, True])
def test_gradient(M, V, C, index, add):
    dout, ids = randn(M, C, seed=C).to(BF), text(M, V, M + V).to(index)
    old = randn(V, C, seed=3).to(BF) if add else None
    check_backward(dout, ids, 1.0, V, old)
    check_backward(dout, ids, torch.tensor(C ** 0.5).float().item(), V, old)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 1024, 1056, 1100, 4099])
@pytest.mark.parametrize("before", [0, 1, 31, 32])
def test_one_row_with_many_tokens(n, before):
    """Runs that begin and end at every place of a chunk, more than 32 whole chunks among them."""
    V, C = 9, 80
    ids = torch.cat((torch.full((before,), 2), torch.full((n,), 5), torch.full((7,), 8))).cuda()
    ids = ids[torch.randperm(ids.numel(), generator=gen(n), device="cuda")]
    check_backward(randn(ids.numel(), C, seed=n).to(BF), ids, 0.5, V)


def test_whole_numbers_are_exact():
    """Sums of whole numbers below 256: exact in every order and chunk, so a token that is missed or counted twice shows."""
    M, V, C = 3000, 40, 64
    ids = torch.randint(-1, V, (M,), generator=gen(4), device="cuda")
    dout = torch.randint(-1, 2, (M, C), generator=gen(5), device="cuda").to(BF)
    ref, _, _ = embedding_backward(dout, ids, 1.0, V)
    assert ref.abs().max() < 256
    assert torch.equal(backward(dout, ids, 1.0, V).double(), ref)
    old = torch.randint(-100, 100, (V, C), generator=gen(6), device="cuda").to(BF)
    assert torch.equal(backward(dout, ids, 1.0, V, old).double(), (ref + old.double()).to(BF).double())


def test_no_token_has_a_row():
    V, C = 700, 96
    dout = randn(50, C, seed=1).to(BF)
    for ids in (torch.full((50,), -1), torch.full((50,), V), torch.full((50,), -(1 << 40)), torch.full((50,), 1 << 40)):
        assert not backward(dout, ids.cuda(), 1.0, V).view(torch.int16).any()
        old = randn(V, C, seed=2).to(BF)
        assert torch.equal(backward(dout, ids.cuda(), 1.0, V, old), old)


def test_ids_past_the_table_give_nan():
    table = randn(10, 32, seed=1).to(BF)
    for index in (torch.int32, torch.int64):
        ids = torch.tensor([0, 10, 9, -1, -7, 2147483647], device="cuda").to(index)
        out = torch.zeros(6, 32, dtype=BF, device="cuda")
        coat.coat_embedding(table, ids, 1.0, out)
        assert out[[1, 5]].isnan().all() and torch.equal(out[[0, 2]], table[[0, 9]]) and not out[[3, 4]].any()


def test_not_a_number_stays_in_its_row():
    V, C = 20, 64
    ids = torch.arange(100, device="cuda") % V
    dout = randn(100, C, seed=1).to(BF)
    dout[3, 5], dout[44, 6] = float("nan"), float("inf")
    got = backward(dout, ids, 1.0, V)
    bad = torch.zeros(V, C, dtype=torch.bool, device="cuda")
    bad[3, 5] = bad[4, 6] = True
    assert torch.equal(~got.isfinite(), bad)


@pytest.mark.parametrize("shift", [8, 16])
def test_pointers_of_16_bytes(shift):
    """Tensors that begin 16 bytes behind a 32-byte boundary, and on one."""
    M, V, C = 100, 60, 80
    ids = text(M, V, 3)

    def view(x):
        t = torch.empty(x.numel() + shift, dtype=BF, device="cuda")[shift:].view(x.shape)
        return t.copy_(x)
    table, dout = view(randn(V, C, seed=1).to(BF)), view(randn(M, C, seed=2).to(BF))
    out, d = view(unwritten(M, C)), view(unwritten(V, C))
    coat.coat_embedding(table, ids, 1.0, out)
    assert torch.equal(out[ids >= 0], table[ids[ids >= 0]])
    ws = workspace(coat.coat_embedding_backward_workspace_bytes(M, V, C))
    coat.coat_embedding_backward(dout, ids, 1.0, d, ws)
    assert torch.equal(d, backward(dout.clone(), ids, 1.0, V))


def test_the_same_bits_every_time():
    M, V, C = 20000, 300, 256
    ids, dout = text(M, V, 1), randn(M, C, seed=1).to(BF)
    first = backward(dout, ids, 0.7, V)
    for _ in range(5):
        assert torch.equal(first, backward(dout, ids, 0.7, V))


def test_many_tokens():
    M, V, C = 300001, 70000, 16
    check_backward(randn(M, C, seed=1).to(BF), text(M, V, 2), 1.0, V)
    check_backward(randn(M, C, seed=1).to(BF), torch.zeros(M, dtype=torch.int32, device="cuda"), 1.0, V)


def test_offsets_past_2_31_elements():
    V, C = 140000, 16384
    ids = torch.tensor([V - 1, 3, V - 1, 131072, 131073], device="cuda")
    table = torch.empty(V, C, dtype=BF, device="cuda")
    table[ids] = randn(5, C, seed=1).to(BF)
    out = unwritten(5, C)
    coat.coat_embedding(table, ids, 1.0, out)
    assert torch.equal(out, table[ids])
    before = table[ids].clone()
    dout = torch.ones(5, C, dtype=BF, device="cuda")
    ws = workspace(coat.coat_embedding_backward_workspace_bytes(5, V, C))
    coat.coat_embedding_backward(dout, ids, 2.0, table, ws)
    want = torch.tensor([4.0, 2.0, 4.0, 2.0, 2.0], device="cuda")
    assert torch.equal(table[ids], want[:, None].expand(5, C).to(BF)) and before.isfinite().all()
    rows = torch.tensor([0, 4, V // 2, V - 2], device="cuda")
    assert not table[rows].any()
    del table


def test_captured_and_replayed_on_another_stream():
    M, V, C = 600, 90, 128
    ids, dout = text(M, V, 1).int(), randn(M, C, seed=1).to(BF)
    table, out, d = randn(V, C, seed=2).to(BF), unwritten(M, C), unwritten(V, C)
    ws = workspace(coat.coat_embedding_backward_workspace_bytes(M, V, C))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        coat.coat_embedding(table, ids, 2.0, out)
        coat.coat_embedding_backward(dout, ids, 2.0, d, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        coat.coat_embedding(table, ids, 2.0, out)
        coat.coat_embedding_backward(dout, ids, 2.0, d, ws)
    for seed in (5, 6):
        ids.copy_(text(M, V, seed))
        dout.copy_(randn(M, C, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, backward(dout, ids, 2.0, V))
        assert torch.equal(out[ids >= 0], (table * 2)[ids[ids >= 0].long()])


def test_differences():
    """The lookup is linear: <dout, out(table + t) - out(table)> = <dtable, t>, within the roundings of both."""
    M, V, C = 500, 70, 64
    ids = text(M, V, 9)
    table, step, dout = (torch.randint(-8, 9, s, generator=gen(i), device="cuda").to(BF)
                         for i, s in enumerate(((V, C), (V, C), (M, C))))
    a, b = unwritten(M, C), unwritten(M, C)
    coat.coat_embedding(table, ids, 0.5, a)
    coat.coat_embedding(table + step, ids, 0.5, b)
    d = backward(dout, ids, 0.5, V).double()
    terms = (d * step.double())
    bound = 2.0 ** -8 * terms.abs().sum()          # a, b are exact: halves of whole numbers up to 16
    assert ((dout.double() * (b.double() - a.double())).sum() - terms.sum()).abs() <= bound


def test_refusals():
    table, out = torch.zeros(8, 32, dtype=BF, device="cuda"), torch.zeros(4, 32, dtype=BF, device="cuda")
    ids, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), workspace(4096)
    with pytest.raises(ValueError, match="out must have"):
        coat.coat_embedding(table, ids, 1.0, out[:3])
    with pytest.raises(TypeError, match="dtype"):
        coat.coat_embedding(table.float(), ids, 1.0, out)
    with pytest.raises(TypeError, match="dtype"):
        coat.coat_embedding(table, ids.short(), 1.0, out)
    with pytest.raises(ValueError, match="contiguous"):
        coat.coat_embedding(table.T.contiguous().T, ids, 1.0, out)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_embedding(table, ids, float("nan"), out)
    with pytest.raises(coat.CoatError, match="INVALID_ARG"):
        coat.coat_embedding_backward(out, ids, 1.0, table, ws[:16])
    with pytest.raises(coat.CoatError, match="MISALIGNED"):
        coat.coat_embedding(table, torch.zeros(5, dtype=torch.int32, device="cuda")[1:], 1.0, out)
    with pytest.raises(TypeError, match="workspace"):
        coat.coat_embedding_backward(out, ids, 1.0, table, ws.cpu())
    assert ws.dtype == U8


def in_order(terms):
    s = torch.zeros_like(terms[0])
    for t in terms:
        s = s + t
    return s


@pytest.mark.parametrize("before,n", [(0, 20), (0, 33), (10, 22), (10, 23), (0, 400), (17, 1000), (31, 5000)])
@pytest.mark.parametrize("add", [False, True])
def test_the_order_of_a_rows_sum(before, n, add):
    """The header's: a row's tokens in their order between cuts at every 32nd of the sorted tokens; then those sums, the first one
    and then every W-th in turn for each of W warps, 4 where the table is written and 2 where it is added to; then the warps'.
    Terms of sizes that differ by 2^12 and cancel, so that what is left is each addition's rounding, float32 for float32 as
    here."""
    C, W = 512, 2 if add else 4
    ids = torch.cat((torch.zeros(before), torch.ones(n))).long().cuda()
    ids = ids[torch.randperm(before + n, generator=gen(n), device="cuda")]
    half = (randn(n - n // 2, C, seed=n) * torch.exp2(12 * torch.rand(n - n // 2, C, generator=gen(n + 1), device="cuda"))).to(BF)
    own = torch.cat((half, -half[:n // 2]))[torch.randperm(n, generator=gen(n + 2), device="cuda")]
    dout = randn(before + n, C, seed=3).to(BF)
    dout[ids == 1] = own
    got = backward(dout, ids, 1.0, 2, torch.zeros(2, C, dtype=BF, device="cuda") if add else None)
    cuts = [0, *range(32 - before % 32, n, 32), n]
    parts = [in_order(own[a:b].float()) for a, b in zip(cuts, cuts[1:])]
    assert len(cuts) == 2 or cuts[1] > 0
    warps = [in_order(parts[:1] * (t == 0) + parts[1 + t::W]) if (t == 0 or parts[1 + t:]) else torch.zeros(C, device="cuda")
             for t in range(W)]
    want = in_order(warps)
    assert torch.equal(got[1], want.to(BF))
