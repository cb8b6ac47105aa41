"""The operators with 8-bit activation checkpoints in float64, from their formulas.

Everything takes and returns float64 tensors (codes as their E4M3 values) on any
device; nothing here calls the library.
"""
import torch


def grid(v):
    """Nearest E4M3 value of v (|v| <= 448), ties to even: steps of 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def quantize(x, G):
    """Values of the codes, scales (a float32 each) and unrounded quotients.  x / S in float64 decides like the exact
    quotient for bf16 x: a quotient that is no midpoint is at least 2^-33 away from one, relatively."""
    parts = x.unflatten(-1, (-1, G))
    S = (parts.abs().amax(-1) / 448).float().double()
    v = (parts / torch.where(S > 0, S, torch.ones_like(S)).unsqueeze(-1)).clamp(-448, 448)
    return grid(v).flatten(-2), S, v.flatten(-2)


def dequantize(val, S, G):
    return val * S.repeat_interleave(G, -1)


def rmsnorm(x, w, eps):
    r = 1 / torch.sqrt(x.square().mean(-1) + eps)
    return x * r.unsqueeze(-1) * w, r


def rmsnorm_backward(dy, xv, r, w):
    """dx, dw (summed over all leading axes), and the sizes of what is added up in them: for error bounds."""
    xh = xv * r.unsqueeze(-1)
    g = dy * w
    c = (g * xh).mean(-1, keepdim=True)
    ca = (g * xh).abs().mean(-1, keepdim=True)
    lead = tuple(range(dy.dim() - 1))
    return (r.unsqueeze(-1) * (g - xh * c), (dy * xh).sum(lead), r.unsqueeze(-1) * (g.abs() + xh.abs() * ca),
            (dy * xh).abs().sum(lead))


def swiglu(g, u):
    return g * torch.special.expit(g) * u


def swiglu_backward(dh, g, u):
    s = torch.special.expit(g)
    return dh * u * s * (1 + g * torch.special.expit(-g)), dh * g * s


def rotate(x, c, s, rot, interleaved):
    """x [M, H, D]; c, s [M, rot/2]."""
    c, s = c.unsqueeze(1), s.unsqueeze(1)
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        out[..., :h], out[..., h:rot] = a * c - b * s, b * c + a * s
    return out


def qk(x, w, eps, c, s, rot, interleaved):
    y, r = rmsnorm(x, w, eps)
    return rotate(y, c, s, rot, interleaved), r


def qk_backward(dy, xv, r, w, c, s, rot, interleaved):
    return rmsnorm_backward(rotate(dy, c, -s, rot, interleaved), xv, r, w)


def weight_grad(dy, xv, row=None, col=None):
    """dW and sum |dy x|, both times |col|."""
    x = xv if row is None else xv * row[:, None]
    dw, size = dy.T @ x, dy.abs().T @ x.abs()
    return (dw, size) if col is None else (dw * col, size * col.abs())
