"""examples/train_mlp_block.py: the operators together.  The block's gradients against autograd
of the same block in 64 bits, and training steps that lower the loss."""
import importlib

import pytest
import torch

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    require_gpu()
    return importlib.import_module("examples.train_mlp_block")


def _reference(block, x, ids, share_coef, activation, z):
    """The block in 64 bits under autograd: (sum of y * weight + balance loss, leaves)."""
    s = block.s
    p = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xr = x.double().requires_grad_()
    normed = torch.nn.functional.layer_norm(xr, (s.width,), p["norm_weight"], p["norm_bias"], 1e-5)
    logits = normed @ p["router"]
    full = torch.softmax(logits, 1)
    y = xr
    for j in range(s.k):
        e = ids[:, j]
        h = torch.einsum("tw,twd->td", normed, p["up"][e])
        g, u = h[:, :s.d], h[:, s.d:]
        if activation == "sparse":
            cut = g.mean(1, keepdim=True) + z * g.std(1, correction=0, keepdim=True)
            a = torch.nn.functional.gelu(torch.relu(g - cut), approximate="tanh") * u
        elif activation == "gelu":
            a = torch.nn.functional.gelu(g, approximate="tanh") * u
        else:
            a = torch.nn.functional.silu(g) * u
        y = y + full.gather(1, e[:, None]) * torch.einsum("td,tdw->tw", a, p["down"][e])
    counts = torch.bincount(ids.reshape(-1), minlength=s.experts).double()
    balance = share_coef * s.experts * (counts / (s.tokens * s.k) * full.mean(0)).sum()
    return y, balance, xr, p


@pytest.mark.parametrize("activation", ["silu", "gelu", "sparse"])
def test_block_gradients_against_autograd(example, activation):
    # bf16 products and an 8-bit checkpoint (half a step of a block of N(0, 1) is about 1% of it;
    # the sparse mask may flip where bf16 products move a gate across the cutoff): the gradients'
    # errors are compared by norm, 4% where nothing flips and 15% where the mask does
    shape = example.Shape(tokens=96, width=64, d=48, experts=4, k=2)
    block = example.Block(shape, activation, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(shape.tokens, shape.width, generator=g, device="cuda").to(torch.bfloat16)
    grad_y = torch.randn(shape.tokens, shape.width, generator=g, device="cuda").to(torch.bfloat16)
    y, loss, saved = block.forward(x)
    up = torch.full((1,), 2.0, device="cuda")
    grad_x, grads = block.backward(grad_y, up, saved)
    ry, rloss, xr, p = _reference(block, x, saved[5], shape.coef, activation, example.Z)
    ((ry * grad_y.double()).sum() + 2 * rloss).backward()

    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    tol = 0.15 if activation == "sparse" else 0.04
    assert off(y, ry.detach()) < 0.02 and off(loss, rloss.detach().view(1)) < 0.01
    assert off(grad_x, xr.grad) < tol
    for name, value in p.items():
        assert off(grads[name], value.grad) < tol, name


@pytest.mark.parametrize("activation", ["silu", "gelu", "sparse"])
def test_training_lowers_the_loss(example, activation):
    losses = example.train(steps=12, activation=activation,
                           shape=example.Shape(tokens=256, width=128, d=64, experts=4))
    assert all(b < a for a, b in zip(losses[:4], losses[1:5])) and losses[-1] < 0.98 * losses[0]
