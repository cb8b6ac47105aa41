"""Cases of the training operators that keep 8-bit activation checkpoints.

Four operators of a transformer block's training step, forward and backward:

* ``norm``    RMS norm (optionally with the residual addition in front), which
              keeps its input as E4M3 codes with one scale per 1 x G group, and
              its backward pass from that checkpoint;
* ``swiglu``  silu(gate) * up with checkpoints of gate and up, and its backward
              pass, which also leaves the product's own checkpoint behind;
* ``qk``      RMS norm of every query and key head with the position rotation,
              with a checkpoint of the heads, and its backward pass;
* ``wgrad``   the weight gradient of a linear layer from its input's checkpoint.

``run`` computes them in plain float32 torch operations, or with the library's
kernels where ``own`` is true.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
EPS = 1e-5
MAX_POS = 4096          # rows of the rotation tables
WORKSPACE = 128 << 20   # bytes of the scratch that a program keeps for its backward calls


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norms of the 7B-shaped model at two sequences of 4096 tokens, residual stream included
        {"name": "norm_fwd_7b", "op": "norm", "back": False, "M": 8192, "N": 4096, "G": 128, "residual": True},
        # a short prompt through the 1B-shaped model: launch latency counts
        {"name": "norm_fwd_short", "op": "norm", "back": False, "M": 33, "N": 2048, "G": 16, "residual": False},
        {"name": "norm_bwd_7b", "op": "norm", "back": True, "M": 8192, "N": 4096, "G": 128, "residual": True},
        # packed documents of the 13B-shaped model: an odd number of tokens, a finer group
        {"name": "norm_bwd_13b_packed", "op": "norm", "back": True, "M": 4099, "N": 5120, "G": 32, "residual": False},
        # the 7B-shaped MLP; gate and up are the halves of one fused projection's output
        {"name": "swiglu_fwd_7b", "op": "swiglu", "back": False, "M": 8192, "N": 11008, "G": 128, "fused": True},
        # a few tokens through the 1B-shaped MLP with separate gate and up
        {"name": "swiglu_fwd_short", "op": "swiglu", "back": False, "M": 17, "N": 8192, "G": 16, "fused": False},
        {"name": "swiglu_bwd_7b", "op": "swiglu", "back": True, "M": 8192, "N": 11008, "G": 128, "fused": True},
        # 32 query and 32 key heads of 128, read from a fused query-key-value projection
        {"name": "qk_fwd_7b", "op": "qk", "back": False, "M": 8192, "Hq": 32, "Hk": 32, "D": 128, "rot": 128,
         "G": 128, "interleaved": False},
        # 40 query heads sharing 10 key heads, an odd number of tokens
        {"name": "qk_bwd_13b_shared", "op": "qk", "back": True, "M": 4101, "Hq": 40, "Hk": 10, "D": 128, "rot": 128,
         "G": 64, "interleaved": False},
        # a handful of tokens, narrow heads, half of each head rotated in adjacent pairs
        {"name": "qk_fwd_short", "op": "qk", "back": False, "M": 3, "Hq": 16, "Hk": 4, "D": 64, "rot": 32,
         "G": 16, "interleaved": True},
        # the 7B-shaped gate projection: its input's checkpoint is the norm's, with the norm's factors
        {"name": "wgrad_7b_gate", "op": "wgrad", "M": 8192, "N": 11008, "K": 4096, "G": 128, "factors": True},
        # a 1B-shaped square projection over an odd, short batch
        {"name": "wgrad_1b_short", "op": "wgrad", "M": 1111, "N": 2048, "K": 2048, "G": 16, "factors": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tokens(rng, hi):
    """Token counts over the whole range: odd ones, and powers of two."""
    m = _log(rng, 1, hi)
    return m | 1 if rng.random() < 0.6 else 1 << (m.bit_length() - 1)


def _width(rng, lo, hi, step):
    """Widths over the whole range: odd multiples of the step, and powers of two."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.4:
        return max(step, 1 << (n.bit_length() - 1))
    return step * ((n // step) | 1)


def draw(rng):
    op = rng.choice(["norm", "norm", "swiglu", "swiglu", "qk", "qk", "wgrad", "wgrad"])
    G = rng.choice([8, 16, 32, 64, 128])
    back = rng.random() < 0.5
    if op == "norm":
        return {"op": op, "back": back, "M": _tokens(rng, 16000), "N": _width(rng, 256, 8000, max(G, 16)), "G": G,
                "residual": rng.random() < 0.5}
    if op == "swiglu":
        return {"op": op, "back": back, "M": _tokens(rng, 8000), "N": _width(rng, 256, 13000, max(G, 16)), "G": G,
                "fused": rng.random() < 0.5}
    if op == "qk":
        Hq, Hk = rng.choice([(1, 1), (5, 1), (7, 7), (16, 2), (32, 4), (32, 32), (40, 10)])
        D = rng.choice([64, 80, 128, 256])
        G = rng.choice([g for g in (8, 16, 32, 64, 128) if D % g == 0])
        rot = rng.choice([D, D, D // 2 // 16 * 16])
        return {"op": op, "back": back, "M": _tokens(rng, 8000 if Hq * D <= 4096 else 4000), "Hq": Hq, "Hk": Hk, "D": D,
                "rot": rot, "G": G, "interleaved": rng.random() < 0.5}
    return {"op": op, "M": _tokens(rng, 8000), "N": _width(rng, 256, 6000, 16), "K": _width(rng, 256, 6000, max(G, 16)),
            "G": G, "factors": rng.random() < 0.5}


def work(case):
    M, G = case["M"], case["G"]
    if case["op"] == "norm":
        N, r = case["N"], 2 if case["residual"] else 0
        if not case["back"]:    # x (and residual) in; y, codes, scales (and h) out
            return {"bytes": M * N * (2 + r + 2 + r + 1 + 4 / G) + 4 * M + 4 * N, "flops": 6 * M * N}
        return {"bytes": M * N * (2 + 1 + 4 / G + r + 2) + 4 * M + 6 * N, "flops": 10 * M * N}
    if case["op"] == "swiglu":
        n = M * case["N"]
        if not case["back"]:    # gate, up in; h and two checkpoints out
            return {"bytes": n * (4 + 2 + 2 + 8 / G), "flops": 10 * n}
        return {"bytes": n * (2 + 2 + 8 / G + 4 + 1 + 4 / G), "flops": 18 * n}
    if case["op"] == "qk":
        H, D = case["Hq"] + case["Hk"], case["D"]
        n = M * H * D
        tables = min(M, MAX_POS) * case["rot"] * 4
        return {"bytes": n * (5 + 4 / G) + 4 * M * H + 4 * M + tables + (16 if not case["back"] else 20) * D,
                "flops": (12 if not case["back"] else 16) * n}
    N, K = case["N"], case["K"]
    extra = 4 * (M + K) if case["factors"] else 0
    return {"bytes": 2 * M * N + M * K * (1 + 4 / G) + 2 * N * K + extra, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activation(gen, M, N):
    """Activations: a scale of its own for each token, a few channels far above the others, one padded token."""
    x = torch.randn(M, N, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=gen, device="cuda"))
    x *= 1 + 20 * (torch.rand(N, generator=gen, device="cuda") < 0.004)
    if M > 8:
        x[M // 2] = 0
    return x.to(torch.bfloat16)


def _gradient(gen, M, N):
    """Gradients: small, with a scale of its own for each token; tokens without a loss have none."""
    g = torch.randn(M, N, generator=gen, device="cuda")
    g *= 1e-3 * torch.exp(torch.randn(M, 1, generator=gen, device="cuda"))
    g[5::97] = 0
    return g.to(torch.bfloat16)


def _norm_weight(gen, N):
    return 1 + 0.1 * torch.randn(N, generator=gen, device="cuda")


def _rstd_of(x):
    return torch.rsqrt(x.float().square().mean(-1) + EPS)


def _positions(gen, M):
    """Positions of packed documents: counting up, starting anew where a document begins."""
    start = torch.rand(M, generator=gen, device="cuda") < 1 / 512
    at = torch.arange(M, device="cuda")
    first = torch.cummax(torch.where(start, at, torch.zeros_like(at)), 0).values
    return ((at - first) % MAX_POS).to(torch.int32)


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    M, G = case["M"], case["G"]
    s = dict(case)
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    if case["op"] == "norm":
        N = case["N"]
        s["weight"] = _norm_weight(gen, N)
        x = _activation(gen, M, N)
        if not case["back"]:
            s["x"] = x
            s["res"] = _activation(gen, M, N) if case["residual"] else None
            s["h"] = _empty(M, N, dtype=bf16) if case["residual"] else None
            s["y"], s["rstd"] = _empty(M, N, dtype=bf16), _empty(M, dtype=f32)
            s["q"], s["scale"] = _empty(M, N, dtype=u8), _empty(M, N // G, dtype=f32)
        else:
            s["q"], s["scale"] = _quantize(x.float(), G)
            s["rstd"] = _rstd_of(x)
            s["dy"] = _gradient(gen, M, N)
            s["dres"] = _gradient(gen, M, N) if case["residual"] else None
            s["dx"], s["dweight"] = _empty(M, N, dtype=bf16), _empty(N, dtype=bf16)
            s["workspace"] = _empty(WORKSPACE, dtype=u8)
    elif case["op"] == "swiglu":
        N = case["N"]
        both = _activation(gen, M, 2 * N)
        if not case["back"]:
            s["gate"], s["up"] = (both[:, :N], both[:, N:]) if case["fused"] else (both[:, :N].contiguous(), both[:, N:].contiguous())
            s["h"] = _empty(M, N, dtype=bf16)
            s["gate_q"], s["up_q"] = _empty(M, N, dtype=u8), _empty(M, N, dtype=u8)
            s["gate_scale"], s["up_scale"] = _empty(M, N // G, dtype=f32), _empty(M, N // G, dtype=f32)
        else:
            s["gate_q"], s["gate_scale"] = _quantize(both[:, :N].float(), G)
            s["up_q"], s["up_scale"] = _quantize(both[:, N:].float(), G)
            s["dh"] = _gradient(gen, M, N)
            if case["fused"]:
                d = _empty(M, 2 * N, dtype=bf16)
                s["dgate"], s["dup"] = d[:, :N], d[:, N:]
            else:
                s["dgate"], s["dup"] = _empty(M, N, dtype=bf16), _empty(M, N, dtype=bf16)
            s["h_q"], s["h_scale"] = _empty(M, N, dtype=u8), _empty(M, N // G, dtype=f32)
    elif case["op"] == "qk":
        Hq, Hk, D, rot = case["Hq"], case["Hk"], case["D"], case["rot"]
        qkv = _activation(gen, M, (Hq + 2 * Hk) * D)
        q = qkv[:, :Hq * D].view(M, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D)
        s["q_weight"], s["k_weight"] = _norm_weight(gen, D), _norm_weight(gen, D)
        angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = _positions(gen, M)
        if not case["back"]:
            s["q"], s["k"] = q, k
            s["q_out"], s["k_out"] = _empty(M, Hq, D, dtype=bf16), _empty(M, Hk, D, dtype=bf16)
            s["q_codes"], s["k_codes"] = _empty(M, Hq, D, dtype=u8), _empty(M, Hk, D, dtype=u8)
            s["q_scale"], s["k_scale"] = _empty(M, Hq, D // G, dtype=f32), _empty(M, Hk, D // G, dtype=f32)
            s["q_rstd"], s["k_rstd"] = _empty(M, Hq, dtype=f32), _empty(M, Hk, dtype=f32)
        else:
            (s["q_codes"], s["q_scale"]), (s["k_codes"], s["k_scale"]) = _quantize(q.float(), G), _quantize(k.float(), G)
            s["q_rstd"], s["k_rstd"] = _rstd_of(q), _rstd_of(k)
            s["dq_out"] = _gradient(gen, M, Hq * D).view(M, Hq, D)
            s["dk_out"] = _gradient(gen, M, Hk * D).view(M, Hk, D)
            d = _empty(M, (Hq + 2 * Hk) * D, dtype=bf16)
            s["dq"], s["dk"] = d[:, :Hq * D].view(M, Hq, D), d[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D)
            s["dq_weight"], s["dk_weight"] = _empty(D, dtype=bf16), _empty(D, dtype=bf16)
            s["workspace"] = _empty(WORKSPACE, dtype=u8)
    else:
        N, K = case["N"], case["K"]
        x = _activation(gen, M, K)
        s["q"], s["scale"] = _quantize(x.float(), G)
        s["dy"] = _gradient(gen, M, N)
        s["row"] = _rstd_of(x) if case["factors"] else None
        s["col"] = _norm_weight(gen, K) if case["factors"] else None
        s["dw"] = _empty(N, K, dtype=bf16)
        s["workspace"] = _empty(WORKSPACE, dtype=u8)
    return s


# ---------------------------------------------------------------------------
# the plain forms, in float32
# ---------------------------------------------------------------------------

def _quantize(x, G):
    """Codes (as bytes) and scales of x [..., N] in groups of G along the last axis."""
    g = x.reshape(*x.shape[:-1], -1, G)
    scale = g.abs().amax(-1) / E4M3_MAX
    y = torch.where(scale[..., None] > 0, g / scale[..., None], 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return y.reshape(x.shape).to(E4M3).view(torch.uint8), scale


def _dequantize(codes, scale, G):
    x = codes.view(E4M3).float()
    return (x.reshape(*x.shape[:-1], -1, G) * scale[..., None]).reshape(x.shape)


def _plain_norm(s):
    G = s["G"]
    if not s["back"]:
        h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(torch.bfloat16)
        x = h.float()
        rstd = 1 / torch.sqrt((x * x).mean(-1) + EPS)
        y = (x * rstd[:, None] * s["weight"]).to(torch.bfloat16)
        codes, scale = _quantize(x, G)
        return _norm_forward_outputs(y, None if s["res"] is None else h, codes, scale, rstd)
    xh = _dequantize(s["q"], s["scale"], G) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xh).sum(0).to(torch.bfloat16)}


def _norm_forward_outputs(y, h, codes, scale, rstd):
    out = {"y": y, "codes": codes.view(E4M3), "scale": scale, "rstd": rstd}
    return out if h is None else {**out, "h": h}


def _plain_swiglu(s):
    G = s["G"]
    if not s["back"]:
        gate, up = s["gate"].float(), s["up"].float()
        h = gate / (1 + torch.exp(-gate)) * up
        (gq, gs), (uq, us) = _quantize(gate, G), _quantize(up, G)
        return {"h": h.to(torch.bfloat16), "gate_codes": gq.view(E4M3), "gate_scale": gs,
                "up_codes": uq.view(E4M3), "up_scale": us}
    gate, up = _dequantize(s["gate_q"], s["gate_scale"], G), _dequantize(s["up_q"], s["up_scale"], G)
    sig = 1 / (1 + torch.exp(-gate))
    dh = s["dh"].float()
    hq, hs = _quantize(gate * sig * up, G)
    return {"dgate": (dh * up * sig * (1 + gate * (1 - sig))).to(torch.bfloat16),
            "dup": (dh * gate * sig).to(torch.bfloat16), "h_codes": hq.view(E4M3), "h_scale": hs}


def _rotate(x, c, s, rot, interleaved):
    """The first `rot` entries of each head turned by the angles with cosines c and sines s, in their pairs."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_qk_side(s, side, c, sn):
    G, rot, inter = s["G"], s["rot"], s["interleaved"]
    weight = s[side + "_weight"]
    if not s["back"]:
        x = s[side].float()
        rstd = 1 / torch.sqrt((x * x).mean(-1) + EPS)
        y = _rotate(x * rstd[..., None] * weight, c, sn, rot, inter)
        codes, scale = _quantize(x, G)
        return {side + "_out": y.to(torch.bfloat16), side + "_codes": codes.view(E4M3), side + "_scale": scale, side + "_rstd": rstd}
    rstd = s[side + "_rstd"][..., None]
    xh = _dequantize(s[side + "_codes"], s[side + "_scale"], G) * rstd
    dn = _rotate(s["d" + side + "_out"].float(), c, -sn, rot, inter)
    g = dn * weight
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return {"d" + side: dx.to(torch.bfloat16), "d" + side + "_weight": (dn * xh).sum((0, 1)).to(torch.bfloat16)}


def _plain_qk(s):
    at = s["positions"].long()
    c, sn = s["cos"][at][:, None], s["sin"][at][:, None]
    return {**_plain_qk_side(s, "q", c, sn), **_plain_qk_side(s, "k", c, sn)}


def _plain_wgrad(s):
    x = _dequantize(s["q"], s["scale"], s["G"])
    if s["row"] is not None:
        x = x * s["row"][:, None]
    dw = s["dy"].float().T @ x
    if s["col"] is not None:
        dw = dw * s["col"]
    return {"dw": dw.to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_norm(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_rmsnorm_ckpt(s["x"], s["weight"], EPS, s["G"], s["y"], s["q"], s["scale"], s["rstd"],
                               residual=s["res"], h=s["h"])
        return _norm_forward_outputs(s["y"], s["h"], s["q"], s["scale"], s["rstd"])
    coat.coat_rmsnorm_ckpt_backward(s["dy"], s["q"], s["scale"], s["rstd"], s["weight"], s["G"], s["dx"],
                                    s["dweight"], s["workspace"], dresidual=s["dres"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_swiglu(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_swiglu_ckpt(s["gate"], s["up"], s["G"], s["h"], s["gate_q"], s["gate_scale"], s["up_q"], s["up_scale"])
        return {"h": s["h"], "gate_codes": s["gate_q"].view(E4M3), "gate_scale": s["gate_scale"],
                "up_codes": s["up_q"].view(E4M3), "up_scale": s["up_scale"]}
    coat.coat_swiglu_ckpt_backward(s["dh"], s["gate_q"], s["gate_scale"], s["up_q"], s["up_scale"], s["G"],
                                   s["dgate"], s["dup"], h_q=s["h_q"], h_scale=s["h_scale"])
    return {"dgate": s["dgate"], "dup": s["dup"], "h_codes": s["h_q"].view(E4M3), "h_scale": s["h_scale"]}


def _own_qk(s):
    import coat_fp8_adamw_gb300 as coat
    if not s["back"]:
        coat.coat_qk_norm_rope_ckpt(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["cos"], s["sin"], s["positions"],
                                    s["G"], s["q_out"], s["q_codes"], s["q_scale"], s["q_rstd"],
                                    s["k_out"], s["k_codes"], s["k_scale"], s["k_rstd"], interleaved=s["interleaved"])
        return {n + e: s[n + e].view(E4M3) if e == "_codes" else s[n + e] for n in "qk" for e in ("_out", "_codes", "_scale", "_rstd")}
    coat.coat_qk_norm_rope_ckpt_backward(s["dq_out"], s["dk_out"], s["q_codes"], s["q_scale"], s["q_rstd"],
                                         s["k_codes"], s["k_scale"], s["k_rstd"], s["q_weight"], s["k_weight"],
                                         s["cos"], s["sin"], s["positions"], s["G"], s["dq"], s["dk"],
                                         s["dq_weight"], s["dk_weight"], s["workspace"], interleaved=s["interleaved"])
    return {n: s[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}


def _own_wgrad(s):
    import coat_fp8_adamw_gb300 as coat
    coat.coat_ckpt_weight_grad(s["dy"], s["q"], s["scale"], s["G"], s["dw"], s["workspace"], row_scale=s["row"], col_scale=s["col"])
    return {"dw": s["dw"]}


_PLAIN = {"norm": _plain_norm, "swiglu": _plain_swiglu, "qk": _plain_qk, "wgrad": _plain_wgrad}
_OWN = {"norm": _own_norm, "swiglu": _own_swiglu, "qk": _own_qk, "wgrad": _own_wgrad}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _grid(v):
    """The E4M3 value nearest to v (float64, |v| <= 448), ties to even: steps of 2^(e-3) from 2^e on, 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _codes64(x, G):
    """The codes' values and the scales of x (float64); a scale is a float32."""
    parts = x.unflatten(-1, (x.shape[-1] // G, G))
    top = parts.abs().max(-1).values
    scale = (top / 448).float().double()
    v = parts / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)
    return _grid(v.clamp(-448, 448)).flatten(-2), top / 448


def _value64(codes, scale, G):
    return codes.view(E4M3).double() * scale.double().repeat_interleave(G, -1)


def _sigmoid64(x):
    return torch.special.expit(x)


def _head64(s, side, phase):
    """One of q and k: complex rotation of the pairs."""
    rot, G = s["rot"], s["G"]

    def turn(x, z):
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if s["interleaved"] else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        out = out.flatten(-2) if s["interleaved"] else out.transpose(-1, -2).flatten(-2)
        return torch.cat((out, x[..., rot:]), -1)

    w = s[side + "_weight"].double()
    if not s["back"]:
        x = s[side].double()
        r = (x.square().mean(-1) + EPS).pow(-0.5)
        codes, scale = _codes64(x, G)
        return {side + "_out": turn(x * w * r.unsqueeze(-1), phase), side + "_codes": codes, side + "_scale": scale, side + "_rstd": r}
    r = s[side + "_rstd"].double().unsqueeze(-1)
    xh = _value64(s[side + "_codes"], s[side + "_scale"], G) * r
    dn = turn(s["d" + side + "_out"].double(), phase.conj())
    inner = (dn * w * xh).mean(-1, keepdim=True)
    return {"d" + side: r * (dn * w - inner * xh), "d" + side + "_weight": torch.einsum("mhd,mhd->d", dn, xh)}


def exact(case, seed):
    s = prepare(case, seed)
    op, G = s["op"], s["G"]
    if op == "norm" and not s["back"]:
        h = s["x"].double()
        if s["res"] is not None:
            # the norm's input is a bf16 tensor: the sum, rounded (the float32 sum of two bf16 values rounds
            # to the same bf16 value as the exact one but where they are 2^15 and more apart)
            h = (h + s["res"].double()).float().to(torch.bfloat16).double()
        r = (h.square().mean(1) + EPS).pow(-0.5)
        codes, scale = _codes64(h, G)
        return _exact_norm(h * s["weight"].double() * r[:, None], codes, scale, r, h if s["res"] is not None else None)
    if op == "norm":
        r = s["rstd"].double()[:, None]
        xh = _value64(s["q"], s["scale"], G) * r
        dy, w = s["dy"].double(), s["weight"].double()
        inner = torch.einsum("mn,mn->m", dy * w, xh)[:, None] / case["N"]
        dx = r * (dy * w - inner * xh)
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": torch.einsum("mn,mn->n", dy, xh)}
    if op == "swiglu" and not s["back"]:
        g, u = s["gate"].double(), s["up"].double()
        (gq, gs), (uq, us) = _codes64(g, G), _codes64(u, G)
        return {"h": g * _sigmoid64(g) * u, "gate_codes": gq, "gate_scale": gs, "up_codes": uq, "up_scale": us}
    if op == "swiglu":
        g, u = _value64(s["gate_q"], s["gate_scale"], G), _value64(s["up_q"], s["up_scale"], G)
        p, dh = _sigmoid64(g), s["dh"].double()
        codes, scale = _codes64(g * p * u, G)
        return {"dgate": dh * u * (p + g * p * _sigmoid64(-g)), "dup": dh * g * p, "h_codes": codes, "h_scale": scale}
    if op == "qk":
        at = s["positions"].long()
        phase = torch.complex(s["cos"].double(), s["sin"].double())[at].unsqueeze(1)
        return {**_head64(s, "q", phase), **_head64(s, "k", phase)}
    x = _value64(s["q"], s["scale"], G)
    if s["row"] is not None:
        x *= s["row"].double()[:, None]
    dw = torch.einsum("mn,mk->nk", s["dy"].double(), x)
    return {"dw": dw if s["col"] is None else dw * s["col"].double()}


def _exact_norm(y, codes, scale, rstd, h):
    out = {"y": y, "codes": codes, "scale": scale, "rstd": rstd}
    return out if h is None else {**out, "h": h}
