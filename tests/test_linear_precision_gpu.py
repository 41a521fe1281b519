"""How exact the products' results are, where the elementwise bounds of tests/linear_ref.py are too
wide to tell: exact logits, small losses, errors in norm, small and large values in fp16.

The errors in norm are held to what rounding the 64-bit result to its type takes off (``own``).  A rounded
operand of a product adds an error of the same relative size, independent of it: a root of two."""
import math

import pytest
import torch

from tests import linear_ref as R
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DTYPES = [BF16, F16]


@pytest.fixture(scope="module")
def ga():
    return require_gpu()


@pytest.fixture(autouse=True)
def no_wait_gave_up(ga):
    yield
    assert ga.device_status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(*shape, seed, scale=1.0):
    return scale * torch.randn(shape, generator=_gen(seed), device="cuda")


def _whole(lo, hi, *shape, seed):
    return torch.randint(lo, hi + 1, shape, generator=_gen(seed), device="cuda").float()


def _rms(x):
    return x.double().square().mean().sqrt().item()


def _own(ref, dtype):
    """What rounding to the type takes off, in norm."""
    return (ref.to(dtype).double() - ref).norm().item()


def _off(got, ref):
    return (got.double() - ref).norm().item()


def _losses(x, w, goal):
    """(loss, lse, largest magnitude of a logit) of each token, in 64 bits."""
    logits = x.double() @ w.double().T
    lse = torch.logsumexp(logits, 1)
    return lse - logits.gather(1, goal[:, None])[:, 0], lse, logits.abs().amax(1)


# ----------------------------------------------------------------- exact logits

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [20, 90, 300])
@pytest.mark.parametrize("k", [64, 1000, 4096, 16384])
@pytest.mark.parametrize("kind", ["one-hot", "zeros", "whole"])
def test_exact_logits(ga, kind, k, tokens, dtype):
    """Logits that fp32 sums hold exactly, in any order: loss and lse are off by fp32's roundings alone."""
    v = 700
    if kind == "one-hot":
        x = torch.zeros(tokens, k, device="cuda")
        x[torch.arange(tokens), torch.randint(k, (tokens,), generator=_gen(1), device="cuda")] = 30
        w = _whole(-64, 64, v, k, seed=2) / 64
    elif kind == "zeros":          # all but the first 32 columns of a row
        x = torch.zeros(tokens, k, device="cuda")
        x[:, :32] = _whole(-3, 3, tokens, 32, seed=1)
        w = _whole(-8, 8, v, k, seed=2) / 8
    else:                          # multiples of 1/8 below 2^15
        x = _whole(-2, 2, tokens, k, seed=1) / 8
        w = _whole(-2, 2, v, k, seed=2)
    x, w = x.to(dtype), w.to(dtype)
    w[1] = w[0]                    # two rows alike: a target and its equal
    goal = torch.randint(v, (tokens,), generator=_gen(3), device="cuda")
    goal[0] = 0
    kept = ga.linear_cross_entropy(x, w, goal)
    loss, lse, most = _losses(x, w, goal)
    # A logit l in powers of two is rounded three times at most on its way (the constant, the product, the
    # difference to the row's maximum), 2^-24 of it each; so are the maximum and what is taken back from it.
    # The sum of exponentials is within R.ARITH of its terms.
    bound = most * 2.0 ** -21 + R.ARITH
    assert ((kept.lse - lse).abs() <= bound).all()
    assert ((kept.loss - loss).abs() <= bound).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [64, 320])
@pytest.mark.parametrize("k", [64, 4096])
def test_small_losses_keep_their_bits(ga, k, tokens, dtype):
    """Confident tokens: losses from 1e-1 down to 1e-12, to a relative error."""
    v = 256
    at = torch.arange(tokens, device="cuda") % 64
    x = torch.zeros(tokens, k, device="cuda")
    x[torch.arange(tokens), at] = 8
    w = _whole(-8, 8, v, k, seed=1) / 64                     # logits within 1
    top = torch.floor(64 + 190 * torch.arange(64, device="cuda") / 63) / 64
    w[torch.arange(64), torch.arange(64)] = top              # but the targets', 8 to 31.75
    x, w = x.to(dtype), w.to(dtype)
    kept = ga.linear_cross_entropy(x, w, at)
    others = x.double() @ w.double().T
    goal = others.gather(1, at[:, None])
    others.scatter_(1, at[:, None], -math.inf)
    loss = torch.log1p(torch.exp(others - goal).sum(1))
    assert loss.max() < 0.5 and loss.min() < 1e-11
    # loss = log1p(s 2^(m - t)): t is rounded to 2^-23 of it (constant and product), a relative error of the
    # power; s and the functions within R.ARITH
    assert ((kept.loss - loss).abs() <= loss * (2.0 ** -22 * goal[:, 0] + R.ARITH)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [60, 500])
@pytest.mark.parametrize("k", [64, 500, 1000, 2048, 4096, 10000, 100001])
def test_losses_in_norm(ga, k, tokens, dtype):
    """Dense rows.  The tensor cores cut fp32 sums off towards 0 after every 16 terms, half a unit of
    the sum on average: over k terms 1.3e-9 k of a logit (24 bits, sums half of the last one on average,
    0.72 for the mantissas' mean inverse).  Sums closed after 512 terms lose 6.6e-7 of theirs, and
    their additions round to 2^-25 each on average, a random walk."""
    v = 2000
    w = _randn(v, k, seed=k, scale=2 * k ** -0.5).to(dtype)
    goal = torch.randint(v, (tokens,), generator=_gen(k + 1), device="cuda")
    x = _randn(tokens, k, seed=k + 2)
    x += 3 * torch.rand(tokens, 1, generator=_gen(k + 3), device="cuda") * w[goal].float()
    x = x.to(dtype)
    kept = ga.linear_cross_entropy(x, w, goal)
    loss, lse, most = _losses(x, w, goal)
    bound = _rms(most) * (1.3e-9 * min(k, 512) + 2.0 ** -25 * (k / 512 + 1) ** 0.5 + 2.0 ** -24)
    assert _rms(kept.lse - lse) <= bound
    assert _rms(kept.loss - loss) <= bound


# ------------------------------------------------------- gradients of the loss

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k", [(30, 200), (64, 200), (200, 200), (256, 200), (400, 200), (1000, 200),
                                      (40, 1024), (40, 1025), (300, 1088), (300, 2500), (700, 5001)])
def test_loss_gradients_in_norm(ga, tokens, k, dtype):
    """Up to 256 tokens nothing but the results' own rounding is seen; past that the weight's
    gradient has its rows' rounding too.  Past k = 1024 the logits are closed sums."""
    v = 3000
    x = _randn(tokens, k, seed=tokens).to(dtype)
    w = _randn(v, k, seed=1, scale=2 * k ** -0.5).to(dtype)
    goal = torch.randint(v, (tokens,), generator=_gen(2), device="cuda")
    gl = 16 * (0.25 + torch.rand(tokens, generator=_gen(3), device="cuda"))
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    y = torch.softmax(x.double() @ w.double().T, 1)
    y[torch.arange(tokens), goal] -= 1
    y *= gl.double()[:, None]
    ref_in, ref_w = y @ w.double(), y.T @ x.double()
    assert _off(gi, ref_in) <= 1.1 * _own(ref_in, dtype)
    assert _off(gw, ref_w) <= (1.1 if tokens <= 256 else 1.5) * _own(ref_w, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [64, 256, 257, 700])
def test_small_slopes_beside_large_ones(ga, tokens, dtype):
    """Slopes over 20 powers of two in one batch.  Every token has its likely token in row 0 and a target
    of its own, whose row of the weight's gradient is its slope times its row, all else below 2^-40
    of the largest slope: each of these rows is right to its own rounding."""
    k, v = 96, 1000
    x = _randn(tokens, k, seed=5)
    x[:, 0] = 8
    w = _randn(v, k, seed=6, scale=0.5 * k ** -0.5)
    w[:, 0] = 0
    w[0] = 0
    w[0, 0] = 4
    x, w = x.to(dtype), w.to(dtype)
    goal = 1 + torch.arange(tokens, device="cuda")
    gl = 4096 * 2.0 ** (-20 * torch.arange(tokens, device="cuda") / tokens)
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    y = torch.softmax(x.double() @ w.double().T, 1)
    y[torch.arange(tokens), goal] -= 1
    y *= gl.double()[:, None]
    ref_in, ref_w = y @ w.double(), y.T @ x.double()
    for ref, got, rows in ((ref_w, gw, goal), (ref_in, gi, slice(None))):
        off = (got.double() - ref)[rows].norm(dim=1)
        own = (ref.to(dtype).double() - ref)[rows].norm(dim=1)
        # y's own error is that of logits of 32, rounded to 2^-22 of it on their way
        assert (off <= 1.1 * own + 32 * 2.0 ** -22 * ref[rows].norm(dim=1)).all()


@pytest.mark.parametrize("tokens", [64, 700])
@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 2.0 ** 12])
@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 9])
def test_sizes_of_rows_and_gradients_in_fp16(ga, size, scale, tokens):
    """The elementwise bounds at rows of all sizes and gradients of all sizes in fp16."""
    k, v = 72, 500
    x = _randn(tokens, k, seed=7, scale=size).to(F16)
    w = (_randn(v, k, seed=8, scale=2 * k ** -0.5) / size).to(F16)
    x[1] = 0                                                  # a row of zeros, whatever its slope
    goal = torch.randint(v, (tokens,), generator=_gen(9), device="cuda")
    gl = scale * (0.25 + torch.rand(tokens, generator=_gen(10), device="cuda"))
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    (ri, bi), (rw, bw) = R.entropy_backward(gl.double(), x.double(), w.double(), goal, F16)
    R.check(gi, ri, bi, "grad_in")
    R.check(gw, rw, bw, "grad_weight")


# ------------------------------------------------------- kernels for few rows

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,d,experts", [
    (16, 72, 3200, 1), (16, 72, 3201, 1), (17, 72, 3200, 1), (8, 72, 3200, 1), (9, 1000, 128, 25), (16, 64, 100, 26),
    (16, 71, 3200, 1), (16, 71, 3329, 1), (17, 71, 500, 1), (3, 71, 9700, 1), (3, 71, 9800, 1), (5, 33, 64, 75),
    (5, 33, 64, 76), (20, 1024, 300, 1), (32, 257, 700, 1)])
def test_borders_between_kernels_of_few_rows(ga, m, k, d, experts, dtype):
    """Both sides of the borders, in rows and in tiles, on 16-byte boundaries (k = 72, 1000, 64, 1024) and off them."""
    x = _randn(experts, m, k, seed=m + k).to(dtype)
    w = _randn(experts, 2 * d, k, seed=d, scale=1.3 * k ** -0.5).to(dtype)
    out = ga.linear_silu_and_mul(x, w)
    for i in range(0, experts, 5):
        ref, bound, *_ = R.forward("silu", x[i].double(), w[i].double(), dtype)
        R.check(out[i], ref, bound, "out")


# ------------------------------------------------- gradients of the projections

def _gated(ga, name, x, w, dy, n_rows=None):
    forward, backward = ((ga.linear_silu_and_mul, ga.linear_silu_and_mul_backward) if name == "silu" else
                         (ga.linear_gelu_and_mul, ga.linear_gelu_and_mul_backward))
    _, kept = forward(x, w, n_rows=n_rows, keep=True)
    return backward(dy, x, w, kept, n_rows=n_rows)


def _exact(name, x, w, dy):
    """(grad_in, grad_weight) in 64 bits."""
    x, w, dy = x.double(), w.double(), dy.double()
    d = w.shape[0] // 2
    h = x @ w.T
    a, slope, _ = R.act(name, h[:, :d])
    rows = torch.cat([dy * h[:, d:] * slope, dy * a], 1)
    return rows @ w, rows.T @ x


# rows, k, d: whole sums, and grad_in's few long ones in shares
SIZES = [(64, 256, 96), (700, 200, 300), (60, 72, 5000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("m,k,d", SIZES)
def test_projection_gradients_in_norm(ga, m, k, d, name, dtype):
    """The results' rounding and that of dg and du."""
    x = _randn(m, k, seed=1).to(dtype)
    w = _randn(2 * d, k, seed=2, scale=1.2 * k ** -0.5).to(dtype)
    dy = _randn(m, d, seed=3).to(dtype)
    for got, ref in zip(_gated(ga, name, x, w, dy), _exact(name, x, w, dy)):
        assert _off(got, ref) <= 1.5 * _own(ref, dtype)


@pytest.mark.parametrize("m,k,d", SIZES)
def test_small_gradients_in_fp16(ga, m, k, d):
    """dg and du around 2^-18, below fp16's normal numbers, where the gradients are normal numbers."""
    dy = _randn(m, d, seed=3, scale=2.0 ** -14).to(F16)
    # u of 2^-4, a weight of 8 for grad_in; u of 2^-2, rows of 8 for grad_weight
    for which, size in ((0, 2.0 ** -4 / 8), (1, 8.0)):
        x = _randn(m, k, seed=1, scale=size * (k ** -0.5 if which == 0 else 1)).to(F16)
        w = _randn(2 * d, k, seed=2, scale=8 if which == 0 else 2.0 ** -5 * k ** -0.5).to(F16)
        ref = _exact("silu", x, w, dy)[which]
        assert _own(ref, F16) <= 2.0 ** -11 * ref.norm()      # the type holds the result
        assert _off(_gated(ga, "silu", x, w, dy)[which], ref) <= 1.5 * _own(ref, F16)


@pytest.mark.parametrize("k,d", [(256, 96), (72, 5000)])
def test_large_gradients_in_fp16(ga, k, d):
    """dg and du past 65504, where the weight's gradient is not."""
    x = _randn(4, k, seed=1, scale=0.004).to(F16)
    w = _randn(2 * d, k, seed=2, scale=5 / 0.004 * k ** -0.5).to(F16)
    dy = _randn(4, d, seed=3, scale=32000).clamp(-60000, 60000).to(F16)
    gi, gw = _gated(ga, "silu", x, w, dy)
    ref_in, ref = _exact("silu", x, w, dy)
    h = x.double() @ w.double().T
    assert (dy.double() * h[:, d:]).abs().max() > 2 * 65504 and ref.abs().max() < 60000
    # Four rows of products of normals: a few large terms are most of a norm, and it matters where their mantissas m
    # in [1, 2) lie.  A rounding is off by 2^-11 / (sqrt(3) m) of the value, root mean square: dg's and du's by up to
    # twice the result's own, together up to sqrt(1 + 4) = 2.24 times it.  (This kernel and its arithmetic in 64 bits
    # with dg and du rounded agree to 1e-3 of that: 1.38 to 1.54 for eight seeds.)
    assert _off(gw, ref) <= 2.25 * _own(ref, F16)
    assert not torch.isnan(gi).any()
    far = ref_in.abs() > 70000
    assert (gi[far].double().sign() == ref_in[far].sign()).all() and torch.isinf(gi[far]).all()
    near = ref_in.abs() < 60000
    assert torch.isfinite(gi[near]).all()


def test_experts_of_different_sizes_in_fp16(ga):
    """Each expert's gradients to their own rounding, beside others 2^20 times as large; what lies behind
    the live rows, and an expert without any, have no part in it."""
    sizes, counts = [2.0 ** -14, 1.0, 2.0 ** 6, 2.0 ** -7, 1.0], [70, 100, 33, 64, 0]
    e, m, k, d = len(sizes), 100, 128, 72
    x = _randn(e, m, k, seed=1).to(F16)
    w = _randn(e, 2 * d, k, seed=2, scale=1.2 * k ** -0.5).to(F16)
    dy = _randn(e, m, d, seed=3)
    for i, s in enumerate(sizes):
        dy[i] *= s
    dy = dy.to(F16)
    for i, n in enumerate(counts):
        x[i, n:] = float("nan")
        dy[i, n:] = 60000
    n_rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    gi, gw = _gated(ga, "gelu", x, w, dy, n_rows)
    for i, n in enumerate(counts):
        ri, rw = _exact("gelu", x[i, :n], w[i], dy[i, :n])
        assert _off(gi[i, :n], ri) <= 1.5 * _own(ri, F16), i
        assert _off(gw[i], rw) <= 1.5 * _own(rw, F16), i


def test_special_gradients_in_fp16(ga):
    """An infinity or a NaN in grad_out reaches its own row of grad_in and its own columns' rows of grad_weight, and
    no others; rows of zeros have gradients of zeros."""
    x = _randn(80, 64, seed=1).to(F16)
    w = _randn(2 * 40, 64, seed=2, scale=0.1).to(F16)
    dy = _randn(80, 40, seed=3).to(F16)
    dy[20] = 0
    clean = _gated(ga, "silu", x, w, dy)
    dy[3, 7], dy[70, 11] = float("inf"), float("nan")
    gi, gw = _gated(ga, "silu", x, w, dy)
    rows = torch.ones(80, dtype=torch.bool, device="cuda")
    rows[[3, 70]] = False
    cols = torch.ones(80, dtype=torch.bool, device="cuda")
    cols[[7, 11, 47, 51]] = False
    assert (gi[20] == 0).all()
    assert not torch.isfinite(gi[~rows]).any() and not torch.isfinite(gw[~cols]).any()
    # the power of two under which dg and du are rounded may follow their largest one, which changes no bit
    # of a normal number
    for got, want, keep in ((gi, clean[0], rows), (gw, clean[1], cols)):
        assert (got[keep] - want[keep]).abs().max() <= 2.0 ** -10 * want[keep].abs().max()
    zero = _gated(ga, "silu", x, w, torch.zeros_like(dy))
    assert not zero[0].any() and not zero[1].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_an_outlier_among_32_columns(ga, dtype):
    """The projections are kept under one scale for 32 columns: beside one of 1000 times their size the other 31
    keep 2^-16 of its size, 1.5% of theirs, in the factors of their gradients, and no more is off."""
    m, k, d = 300, 128, 96
    x = _randn(m, k, seed=1).to(dtype)
    w = _randn(2 * d, k, seed=2, scale=k ** -0.5)
    w[[5, d + 40]] *= 1000
    w = w.to(dtype)
    dy = _randn(m, d, seed=3, scale=1 if dtype == BF16 else 2.0 ** -6).to(dtype)
    got, want = _gated(ga, "silu", x, w, dy), R.backward("silu", dy.double(), x.double(), w.double(), dtype)
    R.check(got[0], *want[0], "grad_in")
    R.check(got[1], *want[1], "grad_weight")
    ref = _exact("silu", x, w, dy)[1]
    off = (got[1].double() - ref).norm(dim=1) / ref.norm(dim=1)
    # columns of blocks without an outlier: half a step of the result and of dg or du
    far = [i for i in range(d) if i // 32 not in (0, 1)]
    assert (off[far + [d + i for i in far]] <= 2 * torch.finfo(dtype).eps / 2).all()
    assert (off <= 0.03 + torch.finfo(dtype).eps).all()


# ------------------------------------------------------------ fp16, used as one

def _step(ga, x, w, head, goal, gl):
    """A gated block, its loss and all gradients."""
    y, kept = ga.linear_gelu_and_mul(x, w, keep=True)
    ce = ga.linear_cross_entropy(y, head, goal)
    gy, ghead = ga.linear_cross_entropy_backward(gl, y, head, goal, ce)
    return (y, ce.loss, ghead) + ga.linear_gelu_and_mul_backward(gy, x, w, kept)


def test_captured_and_overlapping_in_fp16(ga):
    """The passes that find the powers of two, in a graph replayed with larger and smaller inputs than it was captured
    with, and in calls on two streams at once."""
    x = _randn(300, 700, seed=1).to(F16)
    w = _randn(2 * 90, 700, seed=2, scale=700 ** -0.5).to(F16)
    head = _randn(500, 90, seed=3, scale=0.5).to(F16)
    goal = torch.randint(500, (300,), generator=_gen(4), device="cuda")
    goal[::7] = -100
    gl = torch.full((300,), 4.0, device="cuda")
    inputs = [x, (x * 2.0 ** -6), (x * 8)]
    now = x.clone()
    want = []
    for v in inputs:
        now.copy_(v)
        want.append([t.clone() for t in _step(ga, now, w, head, goal, gl)])
    now.copy_(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _step(ga, now, w, head, goal, gl)
    for i in (1, 2, 0, 1):
        now.copy_(inputs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[i])), i
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, _step(ga, inputs[i], w, head, goal, gl)))
    torch.cuda.synchronize()
    for i, result in got:
        assert all(torch.equal(a, b) for a, b in zip(result, want[i]))


def test_many_tokens_in_fp16(ga):
    """More tokens than the first pass has warps, and experts more than SMs."""
    x = _randn(20001, 40, seed=1).to(F16)
    w = _randn(50, 40, seed=2, scale=0.3).to(F16)
    goal = torch.randint(-20, 50, (20001,), generator=_gen(3), device="cuda")
    gl = 64 * torch.rand(20001, generator=_gen(4), device="cuda")
    live = goal >= 0
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    (ri, bi), (rw, bw) = R.entropy_backward(gl[live].double(), x[live].double(), w.double(), goal[live], F16)
    R.check(gi[live], ri, bi, "grad_in")
    R.check(gw, rw, bw, "grad_weight")
    e, m, k, d = 400, 5, 24, 41
    x, w, dy = (_randn(*n, seed=i).to(F16) for i, n in enumerate(((e, m, k), (e, 2 * d, k), (e, m, d))))
    n_rows = torch.arange(e, dtype=torch.int32, device="cuda") % 6
    gi, gw = _gated(ga, "silu", x, w, dy, n_rows)
    for i in range(0, e, 7):
        n = i % 6
        for got, (ref, bound) in zip((gi[i, :n], gw[i]),
                                     R.backward("silu", dy[i, :n].double(), x[i, :n].double(), w[i].double(), F16)):
            R.check(got, ref, bound, f"expert {i}")
