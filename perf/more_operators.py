"""Cases of the operators at the two ends of a language model's training step, and of its dropout.

Three operators, forward and backward:

* ``lce``      softmax cross entropy of a linear layer over a large vocabulary, without the logits being kept:
               loss and log of the softmax's sum per token, and from them the gradients of the layer's input and weight;
* ``embed``    embedding lookup with a scale, and the gradient of the table, written over (an embedding of its own) or
               added to what is there (a table that is the output layer's weight too);
* ``dropout``  dropout with an optional residual addition, its mask drawn from a counter-based generator whenever it is
               needed and stored nowhere.

``run`` computes them in plain float32 torch operations, or with the library's kernels where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100           # the target of a token without a loss
WORKSPACE = 1 << 30     # bytes of the scratch that a program keeps for its calls
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the output layer of the 7B-shaped model at two sequences of 4096 tokens
        {"name": "lce_fwd_7b", "op": "lce", "back": False, "M": 8192, "V": 32000, "C": 4096, "zloss": False, "wide": True},
        # a short packed batch of the 1B-shaped model scored for its loss: the weight's bytes are what counts
        {"name": "lce_fwd_short", "op": "lce", "back": False, "M": 33, "V": 50304, "C": 2048, "zloss": False, "wide": False},
        # the example decoder's own step: a small vocabulary, where latency counts
        {"name": "lce_fwd_small", "op": "lce", "back": False, "M": 2048, "V": 512, "C": 1024, "zloss": False, "wide": True},
        {"name": "lce_bwd_7b", "op": "lce", "back": True, "M": 8192, "V": 32000, "C": 4096, "zloss": False, "wide": True},
        # packed documents of the 1B-shaped model, an odd number of tokens, with a gradient of the log-sum too
        {"name": "lce_bwd_1b_packed", "op": "lce", "back": True, "M": 2051, "V": 50304, "C": 2048, "zloss": True, "wide": False},
        # the 7B-shaped model's embedding of two sequences
        {"name": "embed_fwd_7b", "op": "embed", "back": False, "M": 8192, "V": 32000, "C": 4096, "add": False, "wide": True},
        # a handful of tokens
        {"name": "embed_fwd_short", "op": "embed", "back": False, "M": 17, "V": 50304, "C": 2048, "add": False, "wide": False},
        # the whole table's gradient, most of its rows without a token
        {"name": "embed_bwd_7b", "op": "embed", "back": True, "M": 8192, "V": 32000, "C": 4096, "add": False, "wide": True},
        # the 1B-shaped model's tied table: added to the output layer's gradient
        {"name": "embed_bwd_1b_tied", "op": "embed", "back": True, "M": 16411, "V": 50304, "C": 2048, "add": True, "wide": False},
        # behind a block's projection, with the residual stream
        {"name": "dropout_fwd_7b", "op": "dropout", "back": False, "M": 8192, "C": 4096, "p": 0.1, "residual": True},
        # a few tokens
        {"name": "dropout_fwd_short", "op": "dropout", "back": False, "M": 33, "C": 2048, "p": 0.25, "residual": False},
        # the 13B-shaped model's width, an odd number of tokens
        {"name": "dropout_bwd_13b", "op": "dropout", "back": True, "M": 4099, "C": 5120, "p": 0.1, "residual": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _count(rng, lo, hi):
    """Counts over the whole range: odd ones, and powers of two."""
    m = _log(rng, lo, hi)
    return m | 1 if rng.random() < 0.6 else max(lo, 1 << (m.bit_length() - 1))


def _width(rng, lo, hi):
    """Widths over the whole range: odd multiples of 16, and powers of two."""
    n = _log(rng, lo, hi)
    return 1 << (n.bit_length() - 1) if rng.random() < 0.4 else 16 * ((n // 16) | 1)


def draw(rng):
    op = rng.choice(["lce", "lce", "embed", "embed", "dropout"])
    back = rng.random() < 0.5
    if op == "lce":
        while True:
            M, V, C = _count(rng, 1, 8000), _count(rng, 97, 130000), _width(rng, 128, 5000)
            if M * V * C <= 8192 * 32000 * 4096 and V * C <= 50304 * 5120:
                return {"op": op, "back": back, "M": M, "V": V, "C": C, "zloss": back and rng.random() < 0.5,
                        "wide": rng.random() < 0.5}
    if op == "embed":
        while True:
            M, V, C = _count(rng, 1, 40000), _count(rng, 97, 130000), _width(rng, 64, 5000)
            if M * C <= 8192 * 4096 and V * C <= 32000 * 4096:
                return {"op": op, "back": back, "M": M, "V": V, "C": C, "add": back and rng.random() < 0.5,
                        "wide": rng.random() < 0.5}
    while True:
        M, C = _count(rng, 1, 8000), _width(rng, 64, 8000)
        if M * C <= 8192 * 4096:
            return {"op": op, "back": back, "M": M, "C": C, "p": rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]),
                    "residual": not back and rng.random() < 0.5}


def _distinct(case):
    """The expected number of rows of the table that the ids of a case name."""
    v = np.arange(1, case["V"] + 1, dtype=np.float64)
    p = np.log1p(1 / v) / math.log(case["V"] + 1)
    return float(-np.expm1(case["M"] * np.log1p(-p)).sum())


def work(case):
    M, C = case["M"], case["C"]
    if case["op"] == "lce":
        V = case["V"]
        index = (8 if case["wide"] else 4) * M
        if not case["back"]:    # x, weight and targets in; loss and log-sum out
            return {"bytes": 2 * (M + V) * C + index + 8 * M, "flops": 2 * M * V * C}
        return {"bytes": 4 * (M + V) * C + index + (12 if case["zloss"] else 8) * M, "flops": 6 * M * V * C}
    if case["op"] == "embed":
        index, rows = (8 if case["wide"] else 4) * M, _distinct(case)
        if not case["back"]:
            return {"bytes": 2 * C * (M + rows) + index, "flops": M * C}
        return {"bytes": 2 * C * (M + (2 * rows if case["add"] else case["V"])) + index, "flops": 2 * M * C}
    return {"bytes": M * C * (6 if case["residual"] else 4) + 16, "flops": 2 * M * C}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _gradient(gen, M, C):
    """Gradients: small, with a scale of its own for each token; tokens without a loss have none."""
    g = _randn(gen, M, C) * 1e-3 * torch.exp(_randn(gen, M, 1))
    g[5::97] = 0
    return g.to(BF16)


def _tokens(gen, M, V):
    """Token ids as text has them: the k-th token about 1 / k as often as the first."""
    return (torch.exp(_rand(gen, M) * math.log(V + 1)).long() - 1).clamp(0, V - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    M, C = case["M"], case["C"]
    s = dict(case)
    index = torch.int64 if case.get("wide") else torch.int32
    if case["op"] == "lce":
        V = case["V"]
        s["weight"] = (2 * C ** -0.5 * _randn(gen, V, C)).to(BF16)
        t = _tokens(gen, M, V)
        # hidden states behind the last norm: some tokens are all but certain, most are not
        sure = torch.rand(M, 1, generator=gen, device="cuda").square() * 0.3
        x = _randn(gen, M, C) + sure * C ** 0.5 * s["weight"][t].float()
        s["x"] = x.to(BF16)
        t[_rand(gen, M) < 0.03] = IGNORE        # padding, and the first tokens of documents
        s["targets"] = t.to(index)
        if not case["back"]:
            s["loss"], s["lse"] = _empty(M, dtype=F32), _empty(M, dtype=F32)
        else:
            s["lse"] = _log_sum(s["x"].float() @ s["weight"].float().T)
            valid = t >= 0
            s["dloss"] = valid.float() / valid.sum().clamp_min(1)
            s["dlse"] = 2e-4 * s["lse"] * s["dloss"] if case["zloss"] else None
            s["dx"], s["dweight"] = _empty(M, C, dtype=BF16), _empty(V, C, dtype=BF16)
        s["workspace"] = _empty(WORKSPACE, dtype=U8)
    elif case["op"] == "embed":
        V = case["V"]
        ids = _tokens(gen, M, V)
        if M > 8:
            ids[_rand(gen, M) < 0.01] = -1      # padding
        s["ids"] = ids.to(index)
        s["scale"] = C ** 0.5 if case["add"] or V % 2 else 1.0
        if not case["back"]:
            s["table"] = (0.02 * _randn(gen, V, C)).to(BF16)
            s["out"] = _empty(M, C, dtype=BF16)
        else:
            s["dout"] = _gradient(gen, M, C)
            s["dtable"] = (1e-3 * _randn(gen, V, C)).to(BF16) if case["add"] else _empty(V, C, dtype=BF16)
            s["workspace"] = _empty(WORKSPACE, dtype=U8)
    else:
        s["rng"] = torch.tensor([(int(seed) * 0x9E3779B97F4A7C15 + 1) % (1 << 63), int(seed) * 41 % (1 << 40)], device="cuda")
        s["x"] = _gradient(gen, M, C) if case["back"] else _randn(gen, M, C).to(BF16)
        s["res"] = (3 * _randn(gen, M, C)).to(BF16) if case["residual"] else None
        s["y"] = _empty(M, C, dtype=BF16)
    return s


# ---------------------------------------------------------------------------
# the plain forms, in float32
# ---------------------------------------------------------------------------

def _log_sum(z):
    top = z.amax(-1, keepdim=True)
    return (top + (z - top).exp_().sum(-1, keepdim=True).log()).squeeze(-1)


def _plain_lce(s):
    x, w, t = s["x"].float(), s["weight"].float(), s["targets"].long()
    z = x @ w.T
    valid, at = t >= 0, t.clamp_min(0)[:, None]
    if not s["back"]:
        top = z.amax(-1, keepdim=True)
        low = (z - top).exp().sum(-1).log()
        return {"loss": torch.where(valid, top.squeeze(-1) - z.gather(1, at).squeeze(-1) + low, 0.0), "lse": top.squeeze(-1) + low}
    g = torch.where(valid, s["dloss"], 0.0)
    dz = z.sub_(s["lse"][:, None]).exp_().mul_((g if s["dlse"] is None else g + s["dlse"])[:, None])
    dz.scatter_add_(1, at, -g[:, None])
    return {"dx": (dz @ w).to(BF16), "dweight": (dz.T @ x).to(BF16)}


def _plain_embed(s):
    ids = s["ids"].long()
    valid, at = ids >= 0, ids.clamp_min(0)
    if not s["back"]:
        return {"out": torch.where(valid[:, None], s["table"][at].float() * s["scale"], 0.0).to(BF16)}
    d = torch.where(valid[:, None], s["dout"].float(), 0.0)
    sums = torch.zeros(s["dtable"].shape, device="cuda").index_add_(0, at, d).mul_(s["scale"])
    s["dtable"].copy_(sums + s["dtable"].float() if s["add"] else sums)
    return {"dtable": s["dtable"]}


def _bits(rng, n):
    """The 16 random bits of elements 0 .. n - 1: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) of counter
    (element / 8, rng[1]) and key rng[0], both halves of its four words from the low one up."""
    m = 0xFFFFFFFF
    i = torch.arange((n + 7) // 8, device="cuda")
    k0, k1 = rng[0] & m, rng[0] >> 32 & m
    a, b, c, d = i & m, i >> 32, (rng[1] & m).expand_as(i), (rng[1] >> 32 & m).expand_as(i)
    for _ in range(10):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = v >> 32 & m ^ b ^ k0, v & m, u >> 32 & m ^ d ^ k1, u & m
        k0, k1 = k0 + 0x9E3779B9 & m, k1 + 0xBB67AE85 & m
    w = torch.stack((a, b, c, d), -1)
    return torch.stack((w & 0xFFFF, w >> 16), -1).flatten()[:n]


def _drop(p):
    """Of 65536 draws, how many drop an element."""
    return round(p * 65536)


def _plain_dropout(s):
    keep = (_bits(s["rng"], s["x"].numel()) >= _drop(s["p"])).view(s["x"].shape)
    y = torch.where(keep, s["x"].float() * (65536 / (65536 - _drop(s["p"]))), 0.0)
    return {"dx" if s["back"] else "y": (y if s["res"] is None else y + s["res"].float()).to(BF16)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_lce(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_linear_cross_entropy(s["x"], s["weight"], s["targets"], s["loss"], s["lse"], s["workspace"])
        return {"loss": s["loss"], "lse": s["lse"]}
    coat.coat_linear_cross_entropy_backward(s["x"], s["weight"], s["targets"], s["lse"], s["dloss"], s["dx"], s["dweight"],
                                            s["workspace"], dlse=s["dlse"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_embed(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_embedding(s["table"], s["ids"], s["scale"], s["out"])
        return {"out": s["out"]}
    coat.coat_embedding_backward(s["dout"], s["ids"], s["scale"], s["dtable"], s["workspace"], accumulate=s["add"])
    return {"dtable": s["dtable"]}


def _own_dropout(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_dropout(s["x"], s["p"], s["rng"], s["y"], residual=s["res"])
        return {"y": s["y"]}
    coat.coat_dropout_backward(s["x"], s["p"], s["rng"], s["y"])
    return {"dx": s["y"]}


_PLAIN = {"lce": _plain_lce, "embed": _plain_embed, "dropout": _plain_dropout}
_OWN = {"lce": _own_lce, "embed": _own_embed, "dropout": _own_dropout}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_lce(s):
    x, w, t = s["x"].double(), s["weight"].double(), s["targets"].long()
    one = torch.zeros(t.numel(), w.shape[0], device="cuda", dtype=torch.bool)
    has = (t >= 0).nonzero().squeeze(-1)
    one[has, t[has]] = True
    z = torch.einsum("mc,vc->mv", x, w)
    if not s["back"]:
        lse = torch.logsumexp(z, 1)
        said = one.any(1)
        return {"loss": torch.where(said, lse - torch.where(one, z, torch.zeros_like(z)).sum(1), torch.zeros_like(lse)), "lse": lse}
    g = s["dloss"].double() * one.any(1)
    dz = torch.exp(z - s["lse"].double()[:, None])
    dz = dz * (g if s["dlse"] is None else g + s["dlse"].double())[:, None] - one * g[:, None]
    return {"dx": torch.einsum("mv,vc->mc", dz, w), "dweight": torch.einsum("mv,mc->vc", dz, x)}


def _exact_embed(s):
    ids = s["ids"].long()
    has = (ids >= 0).nonzero().squeeze(-1)
    if not s["back"]:
        out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        out[has] = s["table"].double()[ids[has]] * s["scale"]
        return {"out": out}
    start = s["dtable"].double() if s["add"] else torch.zeros(s["dtable"].shape, device="cuda", dtype=torch.float64)
    return {"dtable": start.index_put((ids[has],), s["dout"].double()[has] * s["scale"], accumulate=True)}


def _exact_dropout(s):
    n = s["x"].numel()
    key, offset = (int(v) for v in s["rng"].cpu())
    counter = np.zeros((4, (n + 7) // 8), dtype=np.uint64)
    counter[0] = np.arange(counter.shape[1], dtype=np.uint64)
    counter[2], counter[3] = offset & 0xFFFFFFFF, offset >> 32
    low, high = np.uint64(0xFFFFFFFF), np.uint64(32)
    for r in range(10):
        keys = [np.uint64(((key >> 32 * j) + r * w) & 0xFFFFFFFF) for j, w in enumerate((0x9E3779B9, 0xBB67AE85))]
        p, q = counter[0] * np.uint64(0xD2511F53), counter[2] * np.uint64(0xCD9E8D57)
        counter = np.stack(((q >> high) ^ counter[1] ^ keys[0], q & low, (p >> high) ^ counter[3] ^ keys[1], p & low))
    draws = np.ascontiguousarray(counter.T.astype("<u4")).view("<u2").reshape(-1)[:n]
    drop = int(math.floor(s["p"] * 65536 + 0.5))
    keep = torch.from_numpy((draws >= drop).astype(np.float64)).cuda().view(s["x"].shape)
    y = keep * s["x"].double() * 65536 / (65536 - drop)
    return {"dx" if s["back"] else "y": y if s["res"] is None else y + s["res"].double()}


def exact(case, seed):
    return {"lce": _exact_lce, "embed": _exact_embed, "dropout": _exact_dropout}[case["op"]](prepare(case, seed))
