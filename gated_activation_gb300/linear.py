"""The matrix products next to the gated activations: gated projections, cross entropy.

Argument marshalling only, as in ``training.py``: every step runs in the CUDA library
behind ``include/gated_act_linear.h``, on ``stream`` (the current one by default), with
no fallback.  Operands are bf16 or fp16 CUDA tensors with contiguous columns; rows may be
strided.  Rows that start on 16-byte boundaries are read in place, others are copied first.
A batch of experts has rows and a weight of its own for each: a stride of 0 over the experts is refused.

The kernels' waits are bounded; one that gave up (after a second: see ``gated_act_linear.h``) leaves its
call's outputs undefined, and ``device_status()`` nonzero.

The functions are the two passes of each operator, not nodes of PyTorch's graph: what they
return requires no gradient, whatever their inputs do.  Under autograd, call them in the
forward and the backward of a ``torch.autograd.Function``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import training as _training


class LinearCheckpoint(NamedTuple):
    """Both projections of the rows, in 16 bits with a scale for each block of 32 of a row.

    A value is off by up to 2^-15 of its block's largest: beside one that is 1000 times the others, these are up
    to 3% off in what their own columns' gradients are computed from.
    """

    codes: torch.Tensor      # int16 [T, 2d], or [E, T, 2d]
    scales: torch.Tensor     # uint8 [T, 2 * ceil(d / 32)], or [E, T, ...]


class CrossEntropy(NamedTuple):
    """Each token's cross entropy, and what its gradient reads."""

    loss: torch.Tensor       # fp32 [T]; 0 at tokens that take no part
    lse: torch.Tensor        # fp32 [T]: log of the sum of the logits' exponentials


def _native():
    return _training._module or _training._native()


# -------------------------------------------------------- gated projections

def linear_silu_and_mul(x: torch.Tensor, weight: torch.Tensor, n_rows: torch.Tensor | None = None,
                        keep: bool = False, out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """``silu(x Wg') * (x Wu')`` [T, d] of ``x`` [T, k] and ``weight`` [2d, k], whose rows
    [0, d) are Wg and [d, 2d) are Wu: silu_and_mul of the linear layer's output, in one kernel.

    A batch of experts has ``x`` [E, T, k] and ``weight`` [E, 2d, k]; ``n_rows`` (int32 [E],
    or [1] for one block), read on the device, holds each one's live row count.  Rows past it have no
    effect, and those of ``out`` are not written.

    ``keep=True`` returns ``(out, LinearCheckpoint)`` for the backward pass.
    """
    return _native().linear_silu_and_mul(x, weight, n_rows, keep, out, stream)


def linear_gelu_and_mul(x: torch.Tensor, weight: torch.Tensor, n_rows: torch.Tensor | None = None,
                        keep: bool = False, out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """``gelu_tanh(x Wg') * (x Wu')``, as linear_silu_and_mul."""
    return _native().linear_gelu_and_mul(x, weight, n_rows, keep, out, stream)


def linear_silu_and_mul_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                 kept: LinearCheckpoint, n_rows: torch.Tensor | None = None,
                                 grad_in: torch.Tensor | None = None,
                                 stream: torch.cuda.Stream | None = None):
    """``(grad_in, grad_weight)`` of linear_silu_and_mul, of x's and weight's shapes and type.

    ``n_rows`` as in the forward pass: rows of grad_in past it are not written (``grad_in=``
    gives the buffer).
    """
    return _native().linear_silu_and_mul_backward(grad_out, x, weight, kept, n_rows, grad_in, stream)


def linear_gelu_and_mul_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                 kept: LinearCheckpoint, n_rows: torch.Tensor | None = None,
                                 grad_in: torch.Tensor | None = None,
                                 stream: torch.cuda.Stream | None = None):
    """``(grad_in, grad_weight)`` of linear_gelu_and_mul, as linear_silu_and_mul_backward."""
    return _native().linear_gelu_and_mul_backward(grad_out, x, weight, kept, n_rows, grad_in, stream)


# ------------------------------------------------------------ cross entropy

def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         stream: torch.cuda.Stream | None = None) -> CrossEntropy:
    """Each token's cross entropy of the logits ``x weight'`` against its target, without the
    logits: ``x`` [T, k], ``weight`` [V, k], ``targets`` [T] int32 or int64, contiguous.

    A token whose target lies outside [0, V) takes no part: its loss and lse are 0, and its
    row of x is not used.
    """
    return _native().linear_cross_entropy(x, weight, targets, stream)


def linear_cross_entropy_backward(grad_loss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                  targets: torch.Tensor, kept: CrossEntropy,
                                  stream: torch.cuda.Stream | None = None):
    """``(grad_in [T, k], grad_weight [V, k])`` at ``grad_loss`` (fp32 [T], contiguous: each
    token's); grad_in is 0 at tokens that take no part."""
    return _native().linear_cross_entropy_backward(grad_loss, x, weight, targets, kept, stream)


__all__ = ["LinearCheckpoint", "CrossEntropy", "linear_silu_and_mul", "linear_gelu_and_mul",
           "linear_silu_and_mul_backward", "linear_gelu_and_mul_backward", "linear_cross_entropy",
           "linear_cross_entropy_backward"]
