"""Training a gated MLP block: 8-bit activation checkpoints, layer norm, balance loss.

Argument marshalling only, as in the package's other bindings: every step runs
in the CUDA library behind ``include/gated_act_training.h``, on ``stream`` (the
current one by default), with no fallback.  The marshalling itself is native
(``csrc/binding.cpp``): it checks the arguments, allocates the outputs, which
belong to the stream that the call launches on, and calls the C ABI.  Inputs
live on the device, or in page-locked host memory that the kernels read in
place.

The functions are the two passes of each operator, not nodes of PyTorch's
graph: what they return requires no gradient, whatever their inputs do.  Under
autograd, call them in the forward and the backward of a
``torch.autograd.Function``.  Rows need columns side by side: a gradient that
was expanded (``sum().backward()`` hands one over) is refused, and goes in as
``grad.contiguous()``.
"""
from __future__ import annotations

import importlib.util
import os
from typing import NamedTuple

import torch

import gated_activation_gb300 as _ga

from . import build as _build


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


_module = None


def _native():
    """The native binding, loaded once."""
    global _module
    if _module is None:
        if not os.path.exists(_build.BINDING):
            raise ImportError(
                f"binding {_build.BINDING} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (no fallback exists)")
        _ga.load_library()
        spec = importlib.util.spec_from_file_location("gated_activation_gb300._lib._training",
                                                      _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_up(Checkpoint, BalanceLoss, _ga._check)
        _module = module
    return _module


# ------------------------------------------------------------- checkpoints

def silu_and_mul_checkpoint(x: torch.Tensor, n_rows: torch.Tensor | None = None,
                            d: int | None = None, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """``silu(gate) * up`` of ``x`` ([M, >=2d] bf16, fp16 or fp32; rows may be
    strided) and the 8-bit checkpoint of x: ``(out [M, d], Checkpoint)``.

    ``n_rows`` (an int32 tensor) is the live row count, read by the kernel;
    rows past it are neither read nor written.
    """
    return (_module or _native()).silu_and_mul_checkpoint(x, n_rows, d, out, stream)


def gelu_and_mul_checkpoint(x: torch.Tensor, n_rows: torch.Tensor | None = None,
                            d: int | None = None, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """``gelu_tanh(gate) * up`` and the checkpoint of x, as silu_and_mul_checkpoint."""
    return (_module or _native()).gelu_and_mul_checkpoint(x, n_rows, d, out, stream)


def gelu_and_mul_sparse_checkpoint(x: torch.Tensor, z: float, d: int | None = None,
                                   out: torch.Tensor | None = None,
                                   stream: torch.cuda.Stream | None = None):
    """The sparse GELU gate of ``x`` and its checkpoint: ``(out [T, d], Checkpoint)``.

    The checkpoint holds gate - cutoff in the gate half, with the mask's sign
    exact, and each row's standard deviation.
    """
    return (_module or _native()).gelu_and_mul_sparse_checkpoint(x, z, d, out, stream)


def silu_and_mul_backward(grad_out: torch.Tensor, kept: Checkpoint,
                          n_rows: torch.Tensor | None = None, recompute: bool = False,
                          stream: torch.cuda.Stream | None = None):
    """The gradient [M, 2d] of silu_and_mul's input at the checkpoint's values.

    ``recompute=True`` returns ``(grad_in, out)`` with the activation's output
    [M, d] computed from the checkpoint too.
    """
    return (_module or _native()).silu_and_mul_backward(grad_out, kept, n_rows, recompute, stream)


def gelu_and_mul_backward(grad_out: torch.Tensor, kept: Checkpoint,
                          n_rows: torch.Tensor | None = None, recompute: bool = False,
                          stream: torch.cuda.Stream | None = None):
    """The gradient of gelu_and_mul's input, as silu_and_mul_backward."""
    return (_module or _native()).gelu_and_mul_backward(grad_out, kept, n_rows, recompute, stream)


def gelu_and_mul_sparse_backward(grad_out: torch.Tensor, kept: Checkpoint, z: float,
                                 recompute: bool = False,
                                 stream: torch.cuda.Stream | None = None):
    """The gradient [T, 2d] of gelu_and_mul_sparse's input, the cutoff's own
    dependence on the row included; ``z`` as in the forward pass."""
    return (_module or _native()).gelu_and_mul_sparse_backward(grad_out, kept, z, recompute, stream)


def checkpoint_values(kept: Checkpoint, dtype: torch.dtype = torch.bfloat16,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The values [M, 2d] that a checkpoint stands for, in bf16 or fp32 (both exact)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("checkpoint values are exact in bfloat16 and float32")
    return (_module or _native()).checkpoint_values(kept, dtype == torch.float32, stream)


# -------------------------------------------------------------- layer norm

def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None):
    """Layer norm of ``x`` ([T, d] bf16, fp16 or fp32; rows may be strided):
    ``(out [T, d], mean [T], rstd [T])``, the statistics in fp32.

    ``weight`` and ``bias`` have x's type or are fp32.
    """
    return (_module or _native()).layer_norm(x, weight, bias, eps, out, stream)


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        stream: torch.cuda.Stream | None = None):
    """``(grad_in [T, d], grad_weight [d], grad_bias [d] or None)`` of layer_norm;
    the parameters' gradients are fp32.  ``bias=False``: no bias gradient."""
    return (_module or _native()).layer_norm_backward(grad_out, x, weight, mean, rstd, bias, stream)


# ------------------------------------------------------------ balance loss

def moe_balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float,
                     live: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> BalanceLoss:
    """The balance loss of a router's ``logits`` ([T, E] bf16, fp16 or fp32) and
    its choices ``ids`` ([T, k] int32 or int64, contiguous), with the per-expert counts.

    ``live`` ([T] bool or uint8): a token that is not live takes no part.  An
    id outside [0, E) is a dropped choice and is not counted.
    """
    return (_module or _native()).moe_balance_loss(logits, ids, coef, live, stream)


def moe_balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, kept: BalanceLoss,
                              live: torch.Tensor | None = None,
                              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient [T, E] of the logits, times ``grad_loss`` (an fp32 tensor of
    one element, read on the device); 0 in the rows that are not live."""
    return (_module or _native()).moe_balance_loss_backward(grad_loss, logits, kept, live, stream)


__all__ = ["Checkpoint", "BalanceLoss", "silu_and_mul_checkpoint", "gelu_and_mul_checkpoint",
           "gelu_and_mul_sparse_checkpoint", "silu_and_mul_backward", "gelu_and_mul_backward",
           "gelu_and_mul_sparse_backward", "checkpoint_values", "layer_norm",
           "layer_norm_backward", "moe_balance_loss", "moe_balance_loss_backward"]
