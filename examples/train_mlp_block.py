"""Training steps of a mixture-of-experts MLP block on the library's operators.

    python examples/train_mlp_block.py [--steps 20] [--activation silu|gelu|sparse|fused]

Layer norm, a router with its balance loss, and experts whose gated activation keeps its
input in 8 bits: the block's forward pass, its backward pass written out, and a plain
gradient step.  The matrix products are PyTorch's, but for those of ``fused``: there the
up projections of all experts, their silu gates and the live row counts are one call of
linear_silu_and_mul, and their gradients one of its backward pass.  What the forward pass keeps of each
expert's activation is the 8-bit checkpoint alone: the activation's output, which the down
projection's weight gradient reads, is computed from it again by the backward pass.  An
expert's rows lie in a buffer of fixed capacity, and the balance loss's per-expert counts
tell the activation how many of them are live.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_activation_gb300 as ga  # noqa: E402

Z = 1.6448536269514722       # the sparse GELU's threshold: 95% of the gates


@dataclass
class Shape:
    tokens: int = 512
    width: int = 256         # the model's
    d: int = 128             # an expert's
    experts: int = 8
    k: int = 2
    coef: float = 1e-2       # of the balance loss


class Block:
    """out = x + sum over the token's experts of p_e * down_e(act(up_e(norm(x))))."""

    def __init__(self, shape: Shape, activation: str = "silu", seed: int = 0, device="cuda"):
        self.s, self.activation = shape, activation
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*size, scale=1.0):
            return (scale * torch.randn(size, generator=g, device=device)).to(torch.bfloat16)

        w, d, e = shape.width, shape.d, shape.experts
        self.params = {
            "norm_weight": torch.ones(w, device=device),
            "norm_bias": torch.zeros(w, device=device),
            "router": normal(w, e, scale=w ** -0.5),
            # as a linear layer has it, rows of outputs, for the fused products
            "up": normal(e, 2 * d, w, scale=w ** -0.5) if activation == "fused"
            else normal(e, w, 2 * d, scale=w ** -0.5),
            "down": normal(e, d, w, scale=d ** -0.5),
        }

    def _activate(self, rows, n_rows):
        if self.activation == "sparse":
            return ga.gelu_and_mul_sparse_checkpoint(rows, Z)
        op = ga.silu_and_mul_checkpoint if self.activation == "silu" else ga.gelu_and_mul_checkpoint
        return op(rows, n_rows=n_rows)

    def _activate_backward(self, grad, kept, n_rows):
        if self.activation == "sparse":
            return ga.gelu_and_mul_sparse_backward(grad, kept, Z, recompute=True)
        op = ga.silu_and_mul_backward if self.activation == "silu" else ga.gelu_and_mul_backward
        return op(grad, kept, n_rows=n_rows, recompute=True)

    def forward(self, x):
        """(output, balance loss [1], what the backward pass reads)."""
        s, p = self.s, self.params
        normed, mean, rstd = ga.layer_norm(x, p["norm_weight"], p["norm_bias"])
        logits = normed @ p["router"]
        ids = torch.topk(logits, s.k, dim=1).indices
        balance = ga.moe_balance_loss(logits, ids, s.coef)
        share = torch.softmax(logits.float(), 1).gather(1, ids)

        # a token's place among the rows of each expert that it chose
        chosen = torch.zeros(s.tokens, s.experts, dtype=torch.int64, device=x.device)
        chosen.scatter_(1, ids, 1)
        place = (chosen.cumsum(0) - 1).gather(1, ids)
        rows = x.new_zeros(s.experts, s.tokens, s.width)
        token = torch.arange(s.tokens, device=x.device)[:, None].expand_as(ids)
        rows[ids, place] = normed[token]

        if self.activation == "fused":
            out, checkpoint = ga.linear_silu_and_mul(rows, p["up"], n_rows=balance.counts, keep=True,
                                                     out=x.new_zeros(s.experts, s.tokens, s.d))
            kept, moved = (out, checkpoint), torch.bmm(out, p["down"])
        else:
            hidden = torch.bmm(rows, p["up"])
            kept, moved = [], x.new_zeros(s.experts, s.tokens, s.width)
            for e in range(s.experts):
                out, checkpoint = self._activate(hidden[e], balance.counts[e:e + 1])
                kept.append(checkpoint)
                moved[e] = self._live(out, balance, e) @ p["down"][e]
        y = x + (moved[ids, place].float() * share[..., None]).sum(1).to(x.dtype)
        return y, balance.loss, (x, normed, mean, rstd, logits, ids, balance, share, place, token,
                                 rows, moved, kept)

    def _live(self, rows, balance, e):
        """Rows past the expert's live ones, which no kernel wrote, as zeros."""
        live = torch.arange(len(rows), device=rows.device) < balance.counts[e]
        return torch.where(live[:, None], rows, torch.zeros_like(rows))

    def backward(self, grad_y, grad_loss, saved):
        """(gradient of x, gradients of the parameters)."""
        s, p = self.s, self.params
        x, normed, mean, rstd, logits, ids, balance, share, place, token, rows, moved, kept = saved
        grads = {"up": torch.empty_like(p["up"]), "down": torch.empty_like(p["down"])}

        # the weighted sum over a token's experts
        per_choice = grad_y[:, None, :].float()
        grad_share = (per_choice * moved[ids, place].float()).sum(2)
        grad_moved = torch.zeros_like(moved)
        grad_moved[ids, place] = (per_choice * share[..., None]).to(x.dtype)

        # the experts
        grad_rows = torch.zeros_like(rows)
        if self.activation == "fused":
            out, checkpoint = kept
            grads["down"] = torch.bmm(out.mT, grad_moved)
            grad_rows, grads["up"] = ga.linear_silu_and_mul_backward(
                torch.bmm(grad_moved, p["down"].mT), rows, p["up"], checkpoint,
                n_rows=balance.counts, grad_in=grad_rows)
        for e in range(0 if self.activation == "fused" else s.experts):
            n = balance.counts[e:e + 1]
            grad_hidden, again = self._activate_backward(grad_moved[e] @ p["down"][e].T, kept[e], n)
            grads["down"][e] = self._live(again, balance, e).T @ grad_moved[e]
            grad_hidden = self._live(grad_hidden, balance, e)
            grads["up"][e] = rows[e].T @ grad_hidden
            grad_rows[e] = grad_hidden @ p["up"][e].T
        grad_normed = grad_rows[ids, place].float().sum(1)

        # the router: its probabilities weigh the experts, and the balance loss
        full = torch.softmax(logits.float(), 1)
        grad_p = torch.zeros_like(full).scatter_(1, ids, grad_share)
        grad_logits = full * (grad_p - (full * grad_p).sum(1, keepdim=True))
        grad_logits += ga.moe_balance_loss_backward(grad_loss, logits, balance).float()
        grad_logits = grad_logits.to(x.dtype)
        grads["router"] = normed.T @ grad_logits
        grad_normed = (grad_normed + (grad_logits @ p["router"].T).float()).to(x.dtype)

        grad_x, grads["norm_weight"], grads["norm_bias"] = ga.layer_norm_backward(
            grad_normed, x, p["norm_weight"], mean, rstd)
        return grad_x + grad_y, grads


def train(steps: int = 20, activation: str = "silu", shape: Shape = Shape(), lr: float = 0.5,
          report=None) -> list[float]:
    """Fits the block to a fixed target; the losses of the steps."""
    block = Block(shape, activation)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(shape.tokens, shape.width, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(shape.tokens, shape.width, generator=g, device="cuda")
    one, losses = torch.ones(1, device="cuda"), []
    for step in range(steps):
        y, balance_loss, saved = block.forward(x)
        error = y.float() - target
        loss = error.square().mean() + balance_loss[0]
        grad_y = (error * (2 / error.numel())).to(torch.bfloat16)
        _, grads = block.backward(grad_y, one, saved)
        for name, value in block.params.items():
            value -= (lr * shape.tokens ** 0.5 * grads[name].float()).to(value.dtype)
        losses.append(loss.item())
        if report:
            report(f"step {step}: loss {losses[-1]:.4f}, balance {balance_loss.item():.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--activation", choices=("silu", "gelu", "sparse", "fused"), default="silu")
    args = ap.parse_args()
    train(args.steps, args.activation, report=print)
