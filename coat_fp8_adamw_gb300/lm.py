"""torch front end of the operators at the two ends of a language model and of dropout.

Embedding lookup and its gradient, softmax cross entropy of a linear layer whose
logits are not kept and its gradients, and dropout whose mask is stored nowhere.
As in the rest of the binding, every tensor is the caller's, the calls run on
``stream`` (default: the current torch stream) and return without synchronizing,
a wrong dtype, shape or device raises here and a non-zero status raises CoatError.
"""
from __future__ import annotations

import torch

from .ckpt import _BF16, _F32, _call, _ptr, _rows, _size, _workspace

_I32, _I64 = torch.int32, torch.int64


def _index(t, M: int, name: str, device):
    """The pointer of a list of M int32 or int64 indexes, and whether they are int64."""
    wide = getattr(t, "dtype", None) is _I64
    return _ptr(t, _I64 if wide else _I32, M, name, device), int(wide)


def _matrix(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape


def coat_embedding(table, ids, scale: float, out, stream=None) -> None:
    """out [M, C] = scale table[ids] for table bf16 [V, C] and ids int32 or int64
    (M of them, any shape); out bf16.  A negative id (padding) gives a row of
    zeros, one of V or more a row of NaN."""
    (V, C), dev, M = _matrix(table, "table"), table.device, ids.numel()
    pid, wide = _index(ids, M, "ids", dev)
    _call("coat_embedding", dev, stream, _ptr(table, _BF16, V * C, "table", dev), pid, wide,
          float(scale), M, V, C, _ptr(out, _BF16, M * C, "out", dev))


def coat_embedding_backward_workspace_bytes(M: int, V: int, C: int, device=None) -> int:
    """Bytes of workspace that coat_embedding_backward needs for M tokens and a table [V, C]."""
    return _size("coat_embedding_backward_workspace_bytes", device, M, V, C)


def coat_embedding_backward(dout, ids, scale: float, dtable, workspace, accumulate: bool = False,
                            stream=None) -> None:
    """Gradient of :func:`coat_embedding`'s table: dtable bf16 [V, C] becomes scale
    times the sums of the rows of dout (bf16 [M, C]) over the tokens of each id, or
    has them added when ``accumulate`` (a table that is the output layer's weight
    too; rows without a token are then left as they are).  Ids outside [0, V) have
    no gradient."""
    (V, C), dev, M = _matrix(dtable, "dtable"), dtable.device, ids.numel()
    pid, wide = _index(ids, M, "ids", dev)
    _call("coat_embedding_backward", dev, stream, _ptr(dout, _BF16, M * C, "dout", dev), pid, wide,
          float(scale), M, V, C, int(bool(accumulate)), _ptr(dtable, _BF16, V * C, "dtable", dev),
          *_workspace(workspace, dev))


def coat_linear_cross_entropy_workspace_bytes(M: int, V: int, device=None) -> int:
    """Bytes of workspace that coat_linear_cross_entropy needs."""
    return _size("coat_linear_cross_entropy_workspace_bytes", device, M, V)


def coat_linear_cross_entropy(x, weight, targets, loss, lse, workspace, stream=None) -> None:
    """Softmax cross entropy of the linear layer x weight^T, whose logits are not
    kept: per token lse = log sum exp(z) and loss = lse - z[target], float32 [M],
    for x bf16 [M, C] (rows at any distance), weight bf16 [V, C] and targets int32
    or int64 [M].  A negative target (a token without one) gives loss 0, one of V
    or more NaN."""
    (M, C), (V, _), dev = _matrix(x, "x"), _matrix(weight, "weight"), x.device
    px, ld = _rows(x, M, C, "x", dev)
    pt, wide = _index(targets, M, "targets", dev)
    _call("coat_linear_cross_entropy", dev, stream, px, ld, _ptr(weight, _BF16, V * C, "weight", dev), pt, wide,
          M, V, C, _ptr(loss, _F32, M, "loss", dev), _ptr(lse, _F32, M, "lse", dev), *_workspace(workspace, dev))


def coat_linear_cross_entropy_backward_workspace_bytes(M: int, V: int, C: int, piece: int = 0, device=None) -> int:
    """Bytes of workspace that coat_linear_cross_entropy_backward needs with pieces of
    ``piece`` rows of the weight (0: as few as leave 512 MiB for a piece)."""
    return _size("coat_linear_cross_entropy_backward_workspace_bytes", device, M, V, C, piece)


def coat_linear_cross_entropy_backward(x, weight, targets, lse, dloss, dx, dweight, workspace, dlse=None,
                                       piece: int = 0, stream=None) -> None:
    """Gradients of :func:`coat_linear_cross_entropy`: with dz = exp(z - lse) (dloss +
    dlse) - [v = target] dloss, rounded to bf16 (an operand of the tensor cores),
    dx bf16 [M, C] = dz weight and dweight bf16 [V, C] = dz^T x.  lse as the forward
    pass left it; dloss and dlse float32 [M], dlse 0 when not given; dloss of a
    token without a target does not count.  The logits are formed again, ``piece`` rows of the weight at a
    time (0: as few pieces as leave 512 MiB for one; rounded up to a multiple of
    256)."""
    (M, C), (V, _), dev = _matrix(x, "x"), _matrix(weight, "weight"), x.device
    px, ld = _rows(x, M, C, "x", dev)
    pt, wide = _index(targets, M, "targets", dev)
    _call("coat_linear_cross_entropy_backward", dev, stream, px, ld, _ptr(weight, _BF16, V * C, "weight", dev), pt, wide,
          _ptr(lse, _F32, M, "lse", dev), _ptr(dloss, _F32, M, "dloss", dev),
          None if dlse is None else _ptr(dlse, _F32, M, "dlse", dev), M, V, C, int(piece),
          _ptr(dx, _BF16, M * C, "dx", dev), _ptr(dweight, _BF16, V * C, "dweight", dev), *_workspace(workspace, dev))


def _rng(t, device):
    return _ptr(t, _I64, 2, "rng", device)


def coat_dropout(x, p: float, rng, y, residual=None, stream=None) -> None:
    """y = keep x 65536 / (65536 - T) (+ residual), T = round(65536 p), halves up:
    dropout of x (bf16, contiguous, any shape) whose mask is drawn from rng, an
    int64 tensor (key, upper half of the counter) on the device, by Philox4x32-10
    and stored nowhere.  Calls that may not share their masks need one that differs
    in either; it is read when the kernel runs, so a captured graph draws new bits
    once it has changed."""
    n, dev = x.numel(), x.device
    _call("coat_dropout", dev, stream, _ptr(x, _BF16, n, "x", dev),
          None if residual is None else _ptr(residual, _BF16, n, "residual", dev), float(p),
          _rng(rng, dev), n, _ptr(y, _BF16, n, "y", dev))


def coat_dropout_backward(dy, p: float, rng, dx, stream=None) -> None:
    """Gradient of :func:`coat_dropout` with the same p and rng: dx = keep dy
    65536 / (65536 - T).  The residual's gradient is dy."""
    n, dev = dy.numel(), dy.device
    _call("coat_dropout_backward", dev, stream, _ptr(dy, _BF16, n, "dy", dev), float(p), _rng(rng, dev), n,
          _ptr(dx, _BF16, n, "dx", dev))
