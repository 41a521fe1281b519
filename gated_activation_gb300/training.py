"""Training a gated MLP block: 8-bit activation checkpoints, layer norm, balance loss.

Argument marshalling only, as in the package's other bindings: every step runs
in the CUDA library behind ``include/gated_act_training.h``, on ``stream`` (the
current one by default), with no fallback.  What a call allocates belongs to
the stream it launches on.  Inputs live on the device, or in page-locked host
memory that the kernels read in place.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

import gated_activation_gb300 as _ga

BLOCK = 32          # elements of one half that share a scale byte


class Checkpoint(NamedTuple):
    """What a forward pass keeps of its input rows [M, 2d] in 8 bits."""

    codes: torch.Tensor                 # int8 [M, 2d]
    scales: torch.Tensor                # uint8 [M, 2 * ceil(d / 32)]
    std: torch.Tensor | None = None     # fp32 [M]: gelu_and_mul_sparse only


class BalanceLoss(NamedTuple):
    """The balance loss of a batch of tokens, and what its gradient reads."""

    loss: torch.Tensor                  # fp32 [1]
    counts: torch.Tensor                # int32 [E]: live choices of each expert
    tokens: torch.Tensor                # int32 [1]: live tokens
    mean_p: torch.Tensor                # fp32 [E]: mean router probability
    k: int
    coef: float


# The current stream's handle without a Stream object around it: these calls
# are a few microseconds long on the host, and that object is two of them.
_current_stream = torch._C._cuda_getCurrentRawStream


def _handle(x: torch.Tensor, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(x.get_device() if x.is_cuda else torch.cuda.current_device())


def _lib():
    return _ga._lib or _ga.load_library()


def _new(shape, dtype: torch.dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An uninitialised tensor where ``like`` lives, owned by ``stream``."""
    if stream is None and like.is_cuda:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not like.is_cuda:
        return torch.empty(shape, dtype=dtype, pin_memory=True)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(nbytes: int, like: torch.Tensor, stream) -> torch.Tensor:
    """Device memory for one call, owned by ``stream``."""
    device = like.device if like.is_cuda else torch.device("cuda", torch.cuda.current_device())
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _reachable(x: torch.Tensor, what: str) -> None:
    if not x.is_cuda and not x.is_pinned():
        raise ValueError(f"{what} must be a CUDA tensor or page-locked host memory "
                         "(the library has no CPU path)")


def _rows(x: torch.Tensor, what: str) -> tuple[int, int, int, int]:
    """(rows, columns, row stride, dtype code) of a 2-D tensor with contiguous columns."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    code = _ga._DTYPE_CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"{what} must be one of {tuple(_ga._DTYPE_CODE)}")
    _reachable(x, what)
    m, n = x.shape
    s0, s1 = x.stride()
    if s1 != 1 and n > 1:
        raise ValueError(f"{what}: columns must be contiguous")
    return m, n, (s0 if m > 1 else n), code


def _flat(x: torch.Tensor, what: str, dtype: torch.dtype, shape: tuple) -> int:
    """The address of a contiguous tensor of that type and shape."""
    if x.dtype != dtype or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {list(shape)}, "
                         f"got {x.dtype} {list(x.shape)}")
    _reachable(x, what)
    return x.data_ptr()


def _count(n_rows: torch.Tensor | None) -> int:
    if n_rows is None:
        return 0
    if n_rows.dtype != torch.int32 or n_rows.numel() < 1:
        raise ValueError("n_rows must be an int32 tensor")
    _reachable(n_rows, "n_rows")
    return n_rows.data_ptr()


def _output(out, shape, like, stream):
    if out is None:
        return _new(shape, like.dtype, like, stream)
    _flat(out, "out", like.dtype, shape)
    return out


# ------------------------------------------------------------- checkpoints

def _checkpoint_rows(x, d, out, stream):
    m, n, stride, code = _rows(x, "input")
    if d is None:
        if n % 2:
            raise ValueError("odd row length: pass d explicitly")
        d = n // 2
    if d < 1 or n < 2 * d:
        raise ValueError("rows are shorter than 2d")
    kept = (_new((m, 2 * d), torch.int8, x, stream),
            _new((m, 2 * -(-d // BLOCK)), torch.uint8, x, stream))
    return m, d, stride, code, _output(out, (m, d), x, stream), kept


def _checkpointed(fn, x, n_rows, d, out, stream):
    m, d, stride, code, out, (codes, scales) = _checkpoint_rows(x, d, out, stream)
    rc = getattr(_lib(), fn)(
        out.data_ptr(), codes.data_ptr(), scales.data_ptr(), x.data_ptr(), m, d, stride, code,
        _count(n_rows), _handle(x, stream))
    _ga._check(fn, rc)
    return out, Checkpoint(codes, scales)


def silu_and_mul_checkpoint(x: torch.Tensor, n_rows: torch.Tensor | None = None,
                            d: int | None = None, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """``silu(gate) * up`` of ``x`` ([M, >=2d] bf16, fp16 or fp32; rows may be
    strided) and the 8-bit checkpoint of x: ``(out [M, d], Checkpoint)``.

    ``n_rows`` (an int32 tensor) is the live row count, read by the kernel;
    rows past it are neither read nor written.
    """
    return _checkpointed("silu_and_mul_checkpoint", x, n_rows, d, out, stream)


def gelu_and_mul_checkpoint(x: torch.Tensor, n_rows: torch.Tensor | None = None,
                            d: int | None = None, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """``gelu_tanh(gate) * up`` and the checkpoint of x, as silu_and_mul_checkpoint."""
    return _checkpointed("gelu_and_mul_checkpoint", x, n_rows, d, out, stream)


def gelu_and_mul_sparse_checkpoint(x: torch.Tensor, z: float, d: int | None = None,
                                   out: torch.Tensor | None = None,
                                   stream: torch.cuda.Stream | None = None):
    """The sparse GELU gate of ``x`` and its checkpoint: ``(out [T, d], Checkpoint)``.

    The checkpoint holds gate - cutoff in the gate half, with the mask's sign
    exact, and each row's standard deviation.
    """
    m, d, stride, code, out, (codes, scales) = _checkpoint_rows(x, d, out, stream)
    std = _new((m,), torch.float32, x, stream)
    rc = _lib().gelu_and_mul_sparse_checkpoint(
        out.data_ptr(), codes.data_ptr(), scales.data_ptr(), std.data_ptr(), x.data_ptr(), m, d,
        stride, float(z), code, _handle(x, stream))
    _ga._check("gelu_and_mul_sparse_checkpoint", rc)
    return out, Checkpoint(codes, scales, std)


def _kept(kept: Checkpoint, m: int, d: int) -> tuple[int, int]:
    return (_flat(kept.codes, "codes", torch.int8, (m, 2 * d)),
            _flat(kept.scales, "scales", torch.uint8, (m, 2 * -(-d // BLOCK))))


def _backward_rows(grad_out, kept, recompute, stream):
    m, d, stride, code = _rows(grad_out, "grad_out")
    codes, scales = _kept(kept, m, d)
    grad_in = _new((m, 2 * d), grad_out.dtype, grad_out, stream)
    out = _new((m, d), grad_out.dtype, grad_out, stream) if recompute else None
    return m, d, stride, code, codes, scales, grad_in, out


def _activation_backward(fn, grad_out, kept, n_rows, recompute, stream):
    m, d, stride, code, codes, scales, grad_in, out = _backward_rows(grad_out, kept, recompute,
                                                                     stream)
    rc = getattr(_lib(), fn)(
        grad_in.data_ptr(), out.data_ptr() if recompute else 0, grad_out.data_ptr(), codes, scales,
        m, d, stride, code, _count(n_rows), _handle(grad_out, stream))
    _ga._check(fn, rc)
    return (grad_in, out) if recompute else grad_in


def silu_and_mul_backward(grad_out: torch.Tensor, kept: Checkpoint,
                          n_rows: torch.Tensor | None = None, recompute: bool = False,
                          stream: torch.cuda.Stream | None = None):
    """The gradient [M, 2d] of silu_and_mul's input at the checkpoint's values.

    ``recompute=True`` returns ``(grad_in, out)`` with the activation's output
    [M, d] computed from the checkpoint too.
    """
    return _activation_backward("silu_and_mul_backward", grad_out, kept, n_rows, recompute, stream)


def gelu_and_mul_backward(grad_out: torch.Tensor, kept: Checkpoint,
                          n_rows: torch.Tensor | None = None, recompute: bool = False,
                          stream: torch.cuda.Stream | None = None):
    """The gradient of gelu_and_mul's input, as silu_and_mul_backward."""
    return _activation_backward("gelu_and_mul_backward", grad_out, kept, n_rows, recompute, stream)


def gelu_and_mul_sparse_backward(grad_out: torch.Tensor, kept: Checkpoint, z: float,
                                 recompute: bool = False,
                                 stream: torch.cuda.Stream | None = None):
    """The gradient [T, 2d] of gelu_and_mul_sparse's input, the cutoff's own
    dependence on the row included; ``z`` as in the forward pass."""
    if kept.std is None:
        raise ValueError("the checkpoint of gelu_and_mul_sparse holds std")
    m, d, stride, code, codes, scales, grad_in, out = _backward_rows(grad_out, kept, recompute,
                                                                     stream)
    std = _flat(kept.std, "std", torch.float32, (m,))
    rc = _lib().gelu_and_mul_sparse_backward(
        grad_in.data_ptr(), out.data_ptr() if recompute else 0, grad_out.data_ptr(), codes, scales,
        std, m, d, stride, float(z), code, _handle(grad_out, stream))
    _ga._check("gelu_and_mul_sparse_backward", rc)
    return (grad_in, out) if recompute else grad_in


def checkpoint_values(kept: Checkpoint, dtype: torch.dtype = torch.bfloat16,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The values [M, 2d] that a checkpoint stands for, in bf16 or fp32 (both exact)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("checkpoint values are exact in bfloat16 and float32")
    if kept.codes.dim() != 2 or kept.codes.shape[1] % 2:
        raise ValueError("codes must be 2-D [M, 2d]")
    m, d = kept.codes.shape[0], kept.codes.shape[1] // 2
    codes, scales = _kept(kept, m, d)
    values = _new((m, 2 * d), dtype, kept.codes, stream)
    rc = _lib().gated_act_checkpoint_values(
        values.data_ptr(), codes, scales, m, d, _ga._DTYPE_CODE[dtype],
        _handle(kept.codes, stream))
    _ga._check("gated_act_checkpoint_values", rc)
    return values


# -------------------------------------------------------------- layer norm

def _params(weight, bias, x, d):
    """(weight address, bias address, dtype code) of the norm's parameters."""
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight must be {x.dtype} or float32")
    w = _flat(weight, "weight", weight.dtype, (d,))
    b = 0 if bias is None else _flat(bias, "bias", weight.dtype, (d,))
    return w, b, _ga._DTYPE_CODE[weight.dtype]


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None):
    """Layer norm of ``x`` ([T, d] bf16, fp16 or fp32; rows may be strided):
    ``(out [T, d], mean [T], rstd [T])``, the statistics in fp32.

    ``weight`` and ``bias`` have x's type or are fp32.
    """
    t, d, stride, code = _rows(x, "input")
    w, b, wcode = _params(weight, bias, x, d)
    out = _output(out, (t, d), x, stream)
    mean, rstd = (_new((t,), torch.float32, x, stream) for _ in range(2))
    rc = _lib().layer_norm(
        out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), x.data_ptr(), w, b, t, d, stride,
        float(eps), code, wcode, _handle(x, stream))
    _ga._check("layer_norm", rc)
    return out, mean, rstd


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        stream: torch.cuda.Stream | None = None):
    """``(grad_in [T, d], grad_weight [d], grad_bias [d] or None)`` of layer_norm;
    the parameters' gradients are fp32.  ``bias=False``: no bias gradient."""
    t, d, stride, code = _rows(x, "input")
    gt, gd, gstride, gcode = _rows(grad_out, "grad_out")
    if (gt, gd, gcode) != (t, d, code):
        raise ValueError("grad_out must have the shape and type of the input")
    w, _, wcode = _params(weight, None, x, d)
    mean_p = _flat(mean, "mean", torch.float32, (t,))
    rstd_p = _flat(rstd, "rstd", torch.float32, (t,))
    lib = _lib()
    grad_in = _new((t, d), x.dtype, x, stream)
    grad_weight = _new((d,), torch.float32, x, stream)
    grad_bias = _new((d,), torch.float32, x, stream) if bias else None
    need = lib.layer_norm_backward_workspace_bytes(t, d)
    ws = _scratch(need, x, stream)
    rc = lib.layer_norm_backward(
        grad_in.data_ptr(), grad_weight.data_ptr(), grad_bias.data_ptr() if bias else 0,
        grad_out.data_ptr(), x.data_ptr(), w, mean_p, rstd_p, t, d, stride, gstride, code, wcode,
        ws.data_ptr(), need, _handle(x, stream))
    _ga._check("layer_norm_backward", rc)
    return grad_in, grad_weight, grad_bias


# ------------------------------------------------------------ balance loss

def _live(live: torch.Tensor | None, t: int) -> int:
    if live is None:
        return 0
    if live.dtype not in (torch.bool, torch.uint8):
        raise TypeError("live must be bool or uint8")
    return _flat(live, "live", live.dtype, (t,))


def moe_balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float,
                     live: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> BalanceLoss:
    """The balance loss of a router's ``logits`` ([T, E] bf16, fp16 or fp32) and
    its choices ``ids`` ([T, k] int32 or int64), with the per-expert counts.

    ``live`` ([T] bool or uint8): a token that is not live takes no part.  An
    id outside [0, E) is a dropped choice and is not counted.
    """
    t, e, stride, code = _rows(logits, "logits")
    if ids.dim() != 2 or ids.shape[0] != t or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be [T, k] int32 or int64")
    k = ids.shape[1]
    ids_p = _flat(ids, "ids", ids.dtype, (t, k))
    live_p = _live(live, t)
    lib = _lib()
    loss, mean_p = (_new((n,), torch.float32, logits, stream) for n in (1, e))
    tokens, counts = (_new((n,), torch.int32, logits, stream) for n in (1, e))
    need = lib.moe_balance_loss_workspace_bytes(t, e)
    ws = _scratch(need, logits, stream)
    rc = lib.moe_balance_loss(
        loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), mean_p.data_ptr(),
        logits.data_ptr(), ids_p, live_p, t, e, k, stride, code, int(ids.dtype == torch.int64),
        float(coef), ws.data_ptr(), need, _handle(logits, stream))
    _ga._check("moe_balance_loss", rc)
    return BalanceLoss(loss, counts, tokens, mean_p, k, float(coef))


def moe_balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, kept: BalanceLoss,
                              live: torch.Tensor | None = None,
                              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient [T, E] of the logits, times ``grad_loss`` (an fp32 tensor of
    one element, read on the device); 0 in the rows that are not live."""
    t, e, stride, code = _rows(logits, "logits")
    if grad_loss.dtype != torch.float32 or grad_loss.numel() != 1:
        raise ValueError("grad_loss must be an fp32 tensor of one element")
    _reachable(grad_loss, "grad_loss")
    counts = _flat(kept.counts, "counts", torch.int32, (e,))
    tokens = _flat(kept.tokens, "tokens", torch.int32, (1,))
    live_p = _live(live, t)
    grad = _new((t, e), logits.dtype, logits, stream)
    rc = _lib().moe_balance_loss_backward(
        grad.data_ptr(), grad_loss.data_ptr(), logits.data_ptr(), counts, tokens, live_p, t, e,
        kept.k, stride, code, kept.coef, _handle(logits, stream))
    _ga._check("moe_balance_loss_backward", rc)
    return grad


__all__ = ["Checkpoint", "BalanceLoss", "silu_and_mul_checkpoint", "gelu_and_mul_checkpoint",
           "gelu_and_mul_sparse_checkpoint", "silu_and_mul_backward", "gelu_and_mul_backward",
           "gelu_and_mul_sparse_backward", "checkpoint_values", "layer_norm",
           "layer_norm_backward", "moe_balance_loss", "moe_balance_loss_backward"]
