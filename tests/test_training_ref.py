"""The 64-bit forms that the training operators are tested against: gradients against
differences of the functions they belong to, the 8-bit format against its definition."""
import pytest
import torch

from tests import training_ref as R


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(*shape, seed):
    return torch.randn(shape, generator=_gen(seed), dtype=torch.float64)


def _difference(f, x, dy, h=1e-5):
    """Gradient of sum(f(x) * dy) by central differences."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view_as(x)
        g.view(-1)[i] = ((f(x + e) - f(x - e)) * dy).sum() / (2 * h)
    return g


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation_gradient_against_differences(name):
    v, dy = _randn(3, 16, seed=1), _randn(3, 8, seed=2)

    def f(v):
        return R.act(name, v[:, :8])[0] * v[:, 8:]

    got = R.act_backward(name, v, dy)
    assert torch.allclose(got["grad"][0], _difference(f, v, dy), atol=1e-8, rtol=1e-7)
    assert torch.allclose(got["out"][0], f(v))


@pytest.mark.parametrize("z", [0.0, 0.7, -0.4])
def test_sparse_gradient_against_differences(z):
    # the cutoff moves with the row: differences of the whole op, away from its kink
    d = 9
    x, dy = _randn(4, 2 * d, seed=3), _randn(4, d, seed=4)

    def f(x):
        delta = R.sparse_stats(x, d, z)[2]
        return R.act("gelu", delta.clamp(min=0))[0] * x[:, d:]

    _, std, delta = R.sparse_stats(x, d, z)
    assert delta.abs().min() > 1e-3
    got = R.sparse_backward(torch.cat([delta, x[:, d:]], 1), dy, std[:, 0], z)
    assert torch.allclose(got["grad"][0], _difference(f, x, dy), atol=1e-8, rtol=1e-7)


def test_layer_norm_gradients_against_differences():
    x, w, b = _randn(4, 7, seed=5), _randn(7, seed=6), _randn(7, seed=7)
    dy, eps = _randn(4, 7, seed=8), 1e-3
    got = R.layer_norm_backward(x, dy, w, eps)

    def norm(x, w, b):
        return R.layer_norm(x, w, b, eps)["out"][0]

    tol = dict(atol=1e-8, rtol=1e-7)
    assert torch.allclose(got["grad"][0], _difference(lambda v: norm(v, w, b), x, dy), **tol)
    assert torch.allclose(got["weight"][0], _difference(lambda v: norm(x, v, b), w, dy), **tol)
    assert torch.allclose(got["bias"][0], _difference(lambda v: norm(x, w, v), b, dy), **tol)


def test_balance_gradient_against_differences():
    logits = _randn(6, 5, seed=9)
    ids = torch.randint(-1, 6, (6, 2), generator=_gen(10))      # dropped choices among them
    live = torch.tensor([1, 1, 0, 1, 1, 0], dtype=torch.uint8)
    got = R.balance(logits, ids, live, 0.3)
    one = torch.ones(1, dtype=torch.float64)
    diff = _difference(lambda v: R.balance(v, ids, live, 0.3)["loss"][0], logits, one)
    assert torch.allclose(got["grad"][0], diff, atol=1e-10, rtol=1e-7)
    assert (got["grad"][0][2] == 0).all() and got["tokens"] == 4
    none = R.balance(logits, ids, torch.zeros(6, dtype=torch.uint8), 0.3)
    assert none["loss"][0] == 0 and (none["grad"][0] == 0).all()


def test_encode_is_the_definition():
    v = _randn(5, 70, seed=11) * torch.exp(20 * _randn(5, 1, seed=12))
    v[1] = 0
    v[2, 3] = float("inf")
    v[3, 40] = float("nan")
    v[4, :32] = 127.5 * 2.0 ** -3                                # rounds past 127: the next scale
    codes, scales = R.encode(v)
    assert scales.shape == (5, 3) and scales[1].tolist() == [0, 0, 0]
    assert scales[2, 0] == 255 and scales[3, 1] == 255 and (codes[2, :32] == 0).all()
    assert scales[4, 0] == 127 - 2 and (codes[4, :32] == 64).all()
    s = R.steps(scales, 70)
    ok = ~torch.isnan(s)
    assert ((codes.double() * s - v).abs()[ok] <= s[ok] / 2).all()
    top = R.blocks(codes.double().abs()).amax(2)
    full = (scales > 0) & (scales < 255)
    assert ((top[full] >= 64) & (top[full] <= 127)).all()
