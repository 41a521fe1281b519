"""The 64-bit forms that the gated projections and the cross entropy are tested against:
gradients against autograd and differences, on the CPU."""
import pytest
import torch

from tests import linear_ref as R

BF16 = torch.bfloat16


def _randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _gated(name, x, w):
    d = len(w) // 2
    h = x @ w.T
    act = torch.nn.functional.silu if name == "silu" else \
        lambda g: torch.nn.functional.gelu(g, approximate="tanh")
    return act(h[:, :d]) * h[:, d:]


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_forms(name):
    x, w, dy = _randn(9, 12, seed=1), _randn(14, 12, seed=2), _randn(9, 7, seed=3)
    out, *_ = R.forward(name, x, w, BF16)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    ref = _gated(name, xr, wr)
    ref.backward(dy)
    assert torch.allclose(out, ref.detach(), rtol=1e-12, atol=1e-12)
    (gi, _), (gw, _) = R.backward(name, dy, x, w, BF16)
    assert torch.allclose(gi, xr.grad, rtol=1e-10, atol=1e-10)
    assert torch.allclose(gw, wr.grad, rtol=1e-10, atol=1e-10)
    for t, grad, other in ((x, gi, w), (w, gw, x)):
        for i in range(0, t.numel(), 11):
            move = torch.zeros(t.numel(), dtype=torch.float64)
            move[i] = 1e-6
            move = move.view(t.shape)
            f = (lambda v: (_gated(name, v, w) * dy).sum()) if t is x else \
                (lambda v: (_gated(name, x, v) * dy).sum())
            diff = (f(t + move) - f(t - move)) / 2e-6
            assert abs(grad.reshape(-1)[i] - diff) < 1e-6 * (1 + abs(diff))


def test_entropy_forms():
    x, w, gl = _randn(6, 10, seed=4), _randn(23, 10, seed=5), _randn(6, seed=6)
    goal = torch.tensor([0, 22, 5, 5, 1, 13])
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss = torch.nn.functional.cross_entropy(xr @ wr.T, goal, reduction="none")
    loss.backward(gl)
    got, _, lse, _, logits, _ = R.entropy(x, w, goal)
    assert torch.allclose(got, loss.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(lse, torch.logsumexp(logits, 1))
    (gi, _), (gw, _) = R.entropy_backward(gl, x, w, goal, BF16)
    assert torch.allclose(gi, xr.grad, rtol=1e-10, atol=1e-10)
    assert torch.allclose(gw, wr.grad, rtol=1e-10, atol=1e-10)
    for i in range(0, w.numel(), 17):
        move = torch.zeros(w.numel(), dtype=torch.float64)
        move[i] = 1e-6
        move = move.view(w.shape)
        f = lambda v: (R.entropy(x, v, goal)[0] * gl).sum()  # noqa: E731
        diff = (f(w + move) - f(w - move)) / 2e-6
        assert abs(gw.reshape(-1)[i] - diff) < 1e-6 * (1 + abs(diff))


def test_bounds_catch_mistakes():
    """A gradient without one of its terms, a neighbour's row and a lost step are outside."""
    x, w, dy = _randn(40, 64, seed=7), _randn(24, 64, seed=8) / 8, _randn(40, 12, seed=9)
    (gi, bi), (gw, bw) = R.backward("silu", dy, x, w, BF16)
    R.check(gi.to(BF16), gi, bi, "grad_in")
    for wrong in (gi.roll(1, 0), gi * 1.1, gi + dy.abs().mean() * w.abs().mean()):
        with pytest.raises(AssertionError):
            R.check(wrong.to(BF16), gi, bi, "grad_in")
    with pytest.raises(AssertionError):
        R.check(((gw - gw[:, :1] * 0.2)).to(BF16), gw, bw, "grad_weight")
