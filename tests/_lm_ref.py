"""The operators at the two ends of a language model and dropout in float64, from their formulas, and what their tests share.

Nothing here calls the library."""
import numpy as np
import torch

U, E = 2.0 ** -8, 2.0 ** -24
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def randn(*shape, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda")


def unwritten(*shape, dtype=BF):
    """Filled with a value that no result has, so that what is not written shows."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.fill_(0xFF) if dtype == U8 else t.fill_(float("nan"))


def workspace(n):
    return torch.full((max(int(n), 16),), 0xFF, dtype=U8, device="cuda")


def near(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    assert over.max().item() <= 0, (f"{what}: {over.max().item():.3e} over the bound at {int(over.argmax())} "
                                    f"(ref {ref.flatten()[over.argmax()]:.6e})")


def bf16_bound(ref):
    return U * (1 + U) * ref.abs() + 2.0 ** -133


def embedding(table, ids, scale):
    ids = ids.long()
    return torch.where((ids >= 0)[:, None], table.double()[ids.clamp_min(0)] * scale, 0.0)


def embedding_backward(dout, ids, scale, V):
    """The gradient, and the sums of its terms' sizes, with the number of terms of each row."""
    ids = ids.long()
    has = ((ids >= 0) & (ids < V)).nonzero().squeeze(1)
    d, at = dout.double()[has] * scale, ids[has]
    zeros = torch.zeros(V, dout.shape[1], dtype=torch.float64, device=dout.device)
    n = torch.bincount(at, minlength=V)
    return zeros.index_add(0, at, d), zeros.index_add(0, at, d.abs()), n


def philox(counter, key):
    """Philox4x32-10 of a counter of four words and a key of two (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(rng, start, n):
    """The 16-bit draws of elements start .. start + n - 1, as int64; rng: (key, offset), unsigned or signed."""
    first, last = start // 8, (start + n - 1) // 8
    key, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in rng)
    i = np.arange(first, last + 1, dtype=np.uint64)
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [i & low, i >> up, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    k = [key & 0xFFFFFFFF, key >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> up) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> up) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    w = np.stack(c, -1)
    both = np.stack((w & np.uint64(0xFFFF), w >> np.uint64(16)), -1).reshape(-1).astype(np.int64)
    return torch.from_numpy(both[start - 8 * first:start - 8 * first + n])


def threshold(p):
    return round(float(np.float32(p)) * 65536)


def linear_cross_entropy(x, w, targets):
    """loss, lse, logits and the sums of the logits' terms' sizes at their largest of every row."""
    z = x.double() @ w.double().T
    size = (x.double().abs() @ w.double().abs().T).amax(1)
    t = targets.long()
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, t.clamp(0, w.shape[0] - 1)[:, None]).squeeze(1)
    loss = torch.where(t < 0, 0.0, lse - zt)
    return torch.where(t >= w.shape[0], float("nan"), loss), lse, z, size


def linear_cross_entropy_backward(x, w, targets, lse, dloss, dlse=None):
    """dx, dw, and per element the sums of the sizes of what is added up: of dz itself, and of its two terms, in which the
    errors of the logits (relative ones of e^(z - lse)) count."""
    x, w, t = x.double(), w.double(), targets.long()
    z, size = x @ w.T, x.abs() @ w.abs().T
    g = torch.where(t >= 0, dloss.double(), 0.0)
    p = (z - lse.double()[:, None]).exp() * (g if dlse is None else g + dlse.double())[:, None]
    dz = p.clone()
    has = (t >= 0).nonzero().squeeze(1)
    dz[has, t[has]] -= g[has]
    return dz @ w, dz.T @ x, dz.abs() @ w.abs(), dz.abs().T @ x.abs(), p, size, z
