"""torch front end of the operators that keep 8-bit activation checkpoints.

RMS norm, silu(gate) * up, the query/key head norm with the position rotation,
and a linear layer's weight gradient from the checkpoint of its input (COAT
review page, section 3: FP8 activations kept for the backward pass).  As in the
rest of the binding, every tensor is the caller's, the calls run on ``stream``
(default: the current torch stream) and return without synchronizing, a wrong
dtype, shape or device raises here and a non-zero status raises CoatError.

A checkpoint of x [M, N] is ``q`` uint8 [M, N] and ``scale`` float32 [M, N/G]
(see :func:`coat_act_quantize_fp8`); it stands for scale * E4M3(q).
"""
from __future__ import annotations

import torch

from . import CoatError, _check, _stream_ptr, lib

_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
_functions = {}


def _ptr(t, dtype, numel: int, name: str, device):
    """The pointer of a contiguous tensor of that dtype and size on ``device``.
    These checks are most of a short call's time on the host, so they are made
    in one expression; _check says what is wrong where they fail."""
    try:
        if (t.dtype is dtype and t.get_device() == device.index and t.is_contiguous()
                and t.numel() == numel):
            return t.data_ptr()
    except AttributeError:
        pass
    return _check(t, dtype, numel, name, device)


def _rows(t, M: int, width: int, name: str, device):
    """A bf16 tensor of M rows of ``width`` elements that lie together, the rows
    at any distance: its pointer and the distance in elements."""
    try:   # the common layouts in one expression, as in _ptr
        if t.dtype is _BF16 and t.get_device() == device.index and t.numel() == M * width:
            st = t.stride()
            if (st[-1] == 1 and t.shape[0] == M
                    and (len(st) == 2 or (len(st) == 3 and st[1] == t.shape[2]))):
                return t.data_ptr(), (st[0] if M > 1 else width)
    except (AttributeError, IndexError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() < 2 or t.shape[0] != M or t.numel() != M * width:
        raise ValueError(f"{name} must hold {M} rows of {width} elements, got {tuple(t.shape)}")
    run = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != run:
            raise ValueError(f"{name}: a row's elements must lie together")
        run *= size
    return t.data_ptr(), (t.stride(0) if M > 1 else width)


def _workspace(t, device):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA tensor")
    if t.device != device:
        raise ValueError(f"workspace is on {t.device}, expected {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _groups(n: int, G: int) -> int:
    return n // G if G > 0 else 0


def _call(name: str, device, stream, *args) -> None:
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    if device.type != "cuda":
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        raw = _stream_ptr(stream)
    if torch._C._cuda_getDevice() == device.index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            st = fn(*args, raw)
    if st != 0:
        raise CoatError(st, name)


def _size(name: str, device, *args) -> int:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(getattr(lib(), name)(*(int(v) for v in args)))


def coat_rmsnorm_ckpt(x, weight, eps: float, G: int, y, q, scale, rstd, residual=None, h=None,
                      stream=None) -> None:
    """RMS norm of the rows of x [M, N] (bf16), or of h = x + residual, with a
    checkpoint of its input: y = h rstd weight (bf16 [M, N]), q and scale the
    checkpoint of h, rstd float32 [M].  weight float32 [N]; h (bf16 [M, N]) is
    written when a residual is given."""
    if x.dim() != 2:
        raise ValueError("x must be a 2-D [M, N] tensor")
    if (residual is None) != (h is None):
        raise ValueError("residual and h come together")
    (M, N), dev = x.shape, x.device
    n = M * N
    _call("coat_rmsnorm_ckpt", dev, stream, _ptr(x, _BF16, n, "x", dev),
          None if residual is None else _ptr(residual, _BF16, n, "residual", dev),
          _ptr(weight, _F32, N, "weight", dev), float(eps), M, N, int(G),
          None if h is None else _ptr(h, _BF16, n, "h", dev), _ptr(y, _BF16, n, "y", dev),
          _ptr(q, _U8, n, "q", dev), _ptr(scale, _F32, _groups(n, G), "scale", dev),
          _ptr(rstd, _F32, M, "rstd", dev))


def coat_rmsnorm_ckpt_backward_workspace_bytes(M: int, N: int, device=None) -> int:
    """Bytes of workspace that coat_rmsnorm_ckpt_backward needs on ``device``."""
    return _size("coat_rmsnorm_ckpt_backward_workspace_bytes", device, M, N)


def coat_rmsnorm_ckpt_backward(dy, q, scale, rstd, weight, G: int, dx, dweight, workspace,
                               dresidual=None, stream=None) -> None:
    """Backward pass of :func:`coat_rmsnorm_ckpt` from its checkpoint: dx bf16
    [M, N] (the gradient of x and of the residual), dweight bf16 [N].
    dresidual (bf16 [M, N]) is the gradient that reaches h past the norm."""
    if dy.dim() != 2:
        raise ValueError("dy must be a 2-D [M, N] tensor")
    (M, N), dev = dy.shape, dy.device
    n = M * N
    _call("coat_rmsnorm_ckpt_backward", dev, stream, _ptr(dy, _BF16, n, "dy", dev),
          _ptr(q, _U8, n, "q", dev), _ptr(scale, _F32, _groups(n, G), "scale", dev),
          _ptr(rstd, _F32, M, "rstd", dev), _ptr(weight, _F32, N, "weight", dev),
          None if dresidual is None else _ptr(dresidual, _BF16, n, "dresidual", dev), M, N, int(G),
          _ptr(dx, _BF16, n, "dx", dev), _ptr(dweight, _BF16, N, "dweight", dev),
          *_workspace(workspace, dev))


def coat_swiglu_ckpt(gate, up, G: int, h, gate_q, gate_scale, up_q, up_scale, stream=None) -> None:
    """h = silu(gate) up (bf16 [M, N]) with checkpoints of gate and up.  gate and
    up are bf16 [M, N] whose rows may be apart (halves of one tensor)."""
    if gate.dim() != 2:
        raise ValueError("gate must be a 2-D [M, N] tensor")
    (M, N), dev = gate.shape, gate.device
    n = M * N
    pg, ld = _rows(gate, M, N, "gate", dev)
    pu, ldu = _rows(up, M, N, "up", dev)
    if ld != ldu:
        raise ValueError(f"gate and up must have the same row stride, got {ld} and {ldu}")
    _call("coat_swiglu_ckpt", dev, stream, pg, pu, ld, M, N, int(G),
          _ptr(h, _BF16, n, "h", dev), _ptr(gate_q, _U8, n, "gate_q", dev),
          _ptr(gate_scale, _F32, _groups(n, G), "gate_scale", dev),
          _ptr(up_q, _U8, n, "up_q", dev),
          _ptr(up_scale, _F32, _groups(n, G), "up_scale", dev))


def coat_swiglu_ckpt_backward(dh, gate_q, gate_scale, up_q, up_scale, G: int, dgate, dup, h_q=None,
                              h_scale=None, stream=None) -> None:
    """Backward pass of :func:`coat_swiglu_ckpt` from its checkpoints: dgate and
    dup bf16 [M, N], whose rows may be apart.  h_q (uint8 [M, N]) and h_scale
    (float32 [M, N/G]), when given, receive the checkpoint of silu(gate) up."""
    if dh.dim() != 2:
        raise ValueError("dh must be a 2-D [M, N] tensor")
    if (h_q is None) != (h_scale is None):
        raise ValueError("h_q and h_scale come together")
    (M, N), dev = dh.shape, dh.device
    n = M * N
    pg, ld = _rows(dgate, M, N, "dgate", dev)
    pu, ldu = _rows(dup, M, N, "dup", dev)
    if ld != ldu:
        raise ValueError(f"dgate and dup must have the same row stride, got {ld} and {ldu}")
    _call("coat_swiglu_ckpt_backward", dev, stream, _ptr(dh, _BF16, n, "dh", dev),
          _ptr(gate_q, _U8, n, "gate_q", dev),
          _ptr(gate_scale, _F32, _groups(n, G), "gate_scale", dev),
          _ptr(up_q, _U8, n, "up_q", dev),
          _ptr(up_scale, _F32, _groups(n, G), "up_scale", dev), M, N, int(G), pg, pu, ld,
          None if h_q is None else _ptr(h_q, _U8, n, "h_q", dev),
          None if h_scale is None else _ptr(h_scale, _F32, _groups(n, G), "h_scale", dev))


def _tables(cos, sin, positions, M: int, D: int, dev):
    if cos.dim() != 2:
        raise ValueError("cos must be a 2-D [max_pos, rot/2] tensor")
    max_pos, half = cos.shape
    return (_ptr(cos, _F32, max_pos * half, "cos", dev),
            _ptr(sin, _F32, max_pos * half, "sin", dev), max_pos, 2 * half,
            _ptr(positions, _I32, M, "positions", dev))


def _heads(t, name: str):
    if t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D [M, heads, D] tensor")
    return t.shape


def _side(side: str, M: int, H: int, D: int, G: int, dev, codes, scale, rstd):
    n = M * H * D
    return (_ptr(codes, _U8, n, f"{side}_codes", dev),
            _ptr(scale, _F32, _groups(n, G), f"{side}_scale", dev),
            _ptr(rstd, _F32, M * H, f"{side}_rstd", dev))


def coat_qk_norm_rope_ckpt(q, k, q_weight, k_weight, eps: float, cos, sin, positions, G: int, q_out,
                           q_codes, q_scale, q_rstd, k_out=None, k_codes=None, k_scale=None,
                           k_rstd=None, interleaved: bool = False, stream=None) -> None:
    """RMS norm of every head of q [M, Hq, D] and k [M, Hk, D] (bf16, the tokens'
    rows at any distance: ranges of one projection's output), the position
    rotation of the normed heads, and a checkpoint of the heads as they came.

    q_weight, k_weight float32 [D]; cos, sin float32 [max_pos, rot/2]; positions
    int32 [M].  q_out bf16 [M, Hq, D], q_codes uint8 [M, Hq, D], q_scale float32
    [M, Hq, D/G], q_rstd float32 [M, Hq], and the same for k.  The first ``rot``
    entries of a head are turned in pairs (i, i + rot/2), or (2i, 2i + 1) when
    ``interleaved``.  k may be None (with k_weight and k's outputs)."""
    M, Hq, D = _heads(q, "q")
    dev = q.device
    pq, q_ld = _rows(q, M, Hq * D, "q", dev)
    pk, k_ld, Hk, pkw, kout = None, 0, 0, None, (None, None, None, None)
    if k is not None:
        Mk, Hk, Dk = _heads(k, "k")
        if (Mk, Dk) != (M, D):
            raise ValueError(f"k must be [{M}, heads, {D}], got {tuple(k.shape)}")
        pk, k_ld = _rows(k, M, Hk * D, "k", dev)
        pkw = _ptr(k_weight, _F32, D, "k_weight", dev)
        kout = (_ptr(k_out, _BF16, M * Hk * D, "k_out", dev),
                *_side("k", M, Hk, D, G, dev, k_codes, k_scale, k_rstd))
    pcos, psin, max_pos, rot, ppos = _tables(cos, sin, positions, M, D, dev)
    _call("coat_qk_norm_rope_ckpt", dev, stream, pq, q_ld, Hq, pk, k_ld, Hk, D,
          _ptr(q_weight, _F32, D, "q_weight", dev), pkw, float(eps), pcos, psin, max_pos, rot, ppos,
          int(bool(interleaved)), M, int(G), _ptr(q_out, _BF16, M * Hq * D, "q_out", dev),
          *_side("q", M, Hq, D, G, dev, q_codes, q_scale, q_rstd), *kout)


def coat_qk_norm_rope_ckpt_backward_workspace_bytes(M: int, D: int, device=None) -> int:
    """Bytes of workspace that coat_qk_norm_rope_ckpt_backward needs on ``device``."""
    return _size("coat_qk_norm_rope_ckpt_backward_workspace_bytes", device, M, D)


def coat_qk_norm_rope_ckpt_backward(dq_out, dk_out, q_codes, q_scale, q_rstd, k_codes, k_scale, k_rstd,
                                    q_weight, k_weight, cos, sin, positions, G: int, dq, dk, dq_weight,
                                    dk_weight, workspace, interleaved: bool = False,
                                    stream=None) -> None:
    """Backward pass of :func:`coat_qk_norm_rope_ckpt` from its checkpoint:
    dq bf16 [M, Hq, D] and dk bf16 [M, Hk, D] (the tokens' rows at any distance:
    ranges of one gradient buffer), dq_weight and dk_weight bf16 [D].  dk_out may
    be None (with everything of k)."""
    M, Hq, D = _heads(dq_out, "dq_out")
    dev = dq_out.device
    pdq, dq_ld = _rows(dq, M, Hq * D, "dq", dev)
    pdko, Hk, kin, pkw, pdk, dk_ld, pdkw = None, 0, (None, None, None), None, None, 0, None
    if dk_out is not None:
        Mk, Hk, Dk = _heads(dk_out, "dk_out")
        if (Mk, Dk) != (M, D):
            raise ValueError(f"dk_out must be [{M}, heads, {D}], got {tuple(dk_out.shape)}")
        pdko = _ptr(dk_out, _BF16, M * Hk * D, "dk_out", dev)
        kin = _side("k", M, Hk, D, G, dev, k_codes, k_scale, k_rstd)
        pkw = _ptr(k_weight, _F32, D, "k_weight", dev)
        pdk, dk_ld = _rows(dk, M, Hk * D, "dk", dev)
        pdkw = _ptr(dk_weight, _BF16, D, "dk_weight", dev)
    pcos, psin, max_pos, rot, ppos = _tables(cos, sin, positions, M, D, dev)
    _call("coat_qk_norm_rope_ckpt_backward", dev, stream,
          _ptr(dq_out, _BF16, M * Hq * D, "dq_out", dev), pdko,
          *_side("q", M, Hq, D, G, dev, q_codes, q_scale, q_rstd), *kin, Hq, Hk, D,
          _ptr(q_weight, _F32, D, "q_weight", dev), pkw, pcos, psin, max_pos, rot, ppos,
          int(bool(interleaved)), M, int(G), pdq, dq_ld, pdk, dk_ld,
          _ptr(dq_weight, _BF16, D, "dq_weight", dev), pdkw, *_workspace(workspace, dev))


def coat_ckpt_weight_grad_workspace_bytes(M: int, N: int, K: int, device=None) -> int:
    """Bytes of workspace that coat_ckpt_weight_grad needs on ``device``."""
    return _size("coat_ckpt_weight_grad_workspace_bytes", device, M, N, K)


def coat_ckpt_weight_grad(dy, q, scale, G: int, dw, workspace, row_scale=None, col_scale=None,
                          stream=None) -> None:
    """Weight gradient of a linear layer from the checkpoint of its input:
    dw bf16 [N, K] = (dy^T X) col_scale, X = row_scale scale E4M3(q) rounded to
    bf16 (the operand of the tensor cores; sums are float32), for dy bf16
    [M, N] (rows at any distance), q uint8 [M, K], scale float32 [M, K/G],
    row_scale float32 [M] and col_scale float32 [K] (1 when not given).  With a
    norm's rstd and weight the checkpoint of the norm's input stands for its
    output."""
    if dy.dim() != 2 or q.dim() != 2:
        raise ValueError("dy [M, N] and q [M, K] must be 2-D")
    (M, N), K, dev = dy.shape, q.shape[1], dy.device
    pdy, ld = _rows(dy, M, N, "dy", dev)
    _call("coat_ckpt_weight_grad", dev, stream, pdy, ld, _ptr(q, _U8, M * K, "q", dev),
          _ptr(scale, _F32, _groups(M * K, G), "scale", dev),
          None if row_scale is None else _ptr(row_scale, _F32, M, "row_scale", dev),
          None if col_scale is None else _ptr(col_scale, _F32, K, "col_scale", dev), M, N, K, int(G),
          _ptr(dw, _BF16, N * K, "dw", dev), *_workspace(workspace, dev))
