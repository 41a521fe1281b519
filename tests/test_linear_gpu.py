"""Gated projections and the cross entropy of a linear layer on the GPU against their 64-bit
forms (tests/linear_ref.py, which derives the bounds)."""
import pytest
import torch

from tests import linear_ref as R
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DTYPES = [BF16, F16]
# rows, k, d: one of everything, below and above a ring step and a tile, rows off 16-byte
# boundaries (k or d not a multiple of 8), several tiles, more tiles than pairs of SMs, sums of 2d long
# enough to be split
GATED = [(1, 1, 1), (1, 64, 128), (3, 7, 5), (2, 72, 40), (17, 130, 33), (64, 64, 256),
         (127, 200, 129), (256, 512, 384), (257, 1101, 271), (300, 96, 2000), (1, 2048, 768),
         (9, 4096, 512), (1100, 264, 1032), (2304, 128, 2304),
         (100, 72, 9001), (30, 200, 4096), (300, 520, 5000)]
# tokens, k, vocabulary
ENTROPY = [(1, 1, 1), (1, 64, 256), (2, 8, 3), (5, 7, 31), (33, 72, 300), (64, 128, 1000),
           (128, 96, 5000), (129, 40, 700), (257, 200, 777), (300, 1001, 4099), (511, 256, 16384), (40, 64, 40001), (700, 136, 8200)]


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


def _strided(x, pad, shift):
    """x with `pad` NaN after each row, and `shift` elements before the first."""
    *lead, m, n = x.shape
    e = lead[0] if lead else 1
    buf = torch.full((shift + e * m * (n + pad),), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[shift:].view(*lead, m, n + pad)
    view[..., :n] = x
    return view[..., :n]


def _ops(ga, name):
    return ((ga.linear_silu_and_mul, ga.linear_silu_and_mul_backward) if name == "silu" else
            (ga.linear_gelu_and_mul, ga.linear_gelu_and_mul_backward))


def _operands(m, k, d, dtype, seed, experts=None):
    lead = () if experts is None else (experts,)
    x = _randn(*lead, m, k, seed=seed).to(dtype)
    w = _randn(*lead, 2 * d, k, seed=seed + 1, scale=1.3 * k ** -0.5).to(dtype)
    dy = _randn(*lead, m, d, seed=seed + 2).to(dtype)
    return x, w, dy


def _check_gated(name, x, w, dy, out, grads, dtype):
    ref, bound, *_ = R.forward(name, x.double(), w.double(), dtype)
    R.check(out, ref, bound, "out")
    if grads is not None:
        want = R.backward(name, dy.double(), x.double(), w.double(), dtype)
        for got, (ref, bound), what in zip(grads, want, ("grad_in", "grad_weight")):
            R.check(got, ref, bound, what)


# ------------------------------------------------------------- gated projections

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("m,k,d", GATED)
def test_gated(ga, name, m, k, d, dtype):
    x, w, dy = _operands(m, k, d, dtype, m + k + d)
    forward, backward = _ops(ga, name)
    _check_gated(name, x, w, dy, forward(x, w), None, dtype)
    out, kept = forward(x, w, keep=True)
    _check_gated(name, x, w, dy, out, backward(dy, x, w, kept), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (3, 5), (0, 1)])
@pytest.mark.parametrize("experts", [None, 3])
def test_gated_strides(ga, pad, shift, dtype, experts):
    x, w, dy = _operands(130, 80, 72, dtype, 5, experts)
    forward, backward = _ops(ga, "silu")
    out, kept = forward(x, w, keep=True)
    grads = backward(dy, x, w, kept)
    xs, ws, dys = (_strided(t, pad, shift) for t in (x, w, dy))
    got, again = forward(xs, ws, keep=True)
    assert torch.equal(got, out) and torch.equal(again.codes, kept.codes)
    for a, b in zip(backward(dys, xs, ws, again), grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pad,shift", [(8, 8), (3, 5)])
def test_experts_strides(ga, pad, shift):
    """Rows apart, on 16-byte boundaries and off them, of which the last step is partly live."""
    x, w, dy = _operands(200, 104, 40, BF16, 77, 3)
    counts = torch.tensor([200, 70, 129], dtype=torch.int32, device="cuda")
    xs, ws, dys = _strided(x, pad, shift), _strided(w, pad, shift), _strided(dy, pad, shift)
    want, kept = ga.linear_silu_and_mul(x, w, n_rows=counts, keep=True)
    grads = ga.linear_silu_and_mul_backward(dy, x, w, kept, n_rows=counts)
    got, again = ga.linear_silu_and_mul(xs, ws, n_rows=counts, keep=True)
    others = ga.linear_silu_and_mul_backward(dys, xs, ws, again, n_rows=counts)
    assert torch.equal(grads[1], others[1])
    for i, n in enumerate(counts.tolist()):
        assert torch.equal(want[i, :n], got[i, :n]) and torch.equal(grads[0][i, :n], others[0][i, :n])
        _check_gated("silu", x[i, :n], w[i], dy[i, :n], want[i, :n], (grads[0][i, :n], grads[1][i]), BF16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("m,k,d,counts", [
    (40, 64, 96, [40, 0, 1, 17]), (300, 72, 136, [300, 64, 0, 0, 257, 1, 63, 65]),
    (60, 72, 5000, [60, 0, 33]), (8, 128, 40, [0, 0, 0]), (64, 33, 7, [64, 5]), (100, 64, 64, [-3, 1000, 50]),
    (2, 64, 32, [1 + i % 2 for i in range(200)])])
def test_experts(ga, name, m, k, d, counts, dtype):
    e = len(counts)
    live = [min(max(n, 0), m) for n in counts]
    x, w, dy = _operands(m, k, d, dtype, m + k, e)
    for i, n in enumerate(live):              # what lies past the live rows has no effect
        x[i, n:] = float("nan")
        dy[i, n:] = float("inf")
    n_rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    forward, backward = _ops(ga, name)
    out = torch.full((e, m, d), -7.0, dtype=dtype, device="cuda")
    grad_in = torch.full((e, m, k), -7.0, dtype=dtype, device="cuda")
    got, kept = forward(x, w, n_rows=n_rows, keep=True, out=out)
    assert got.data_ptr() == out.data_ptr()
    gi, gw = backward(dy, x, w, kept, n_rows=n_rows, grad_in=grad_in)
    assert gi.data_ptr() == grad_in.data_ptr()
    for i, n in enumerate(live):
        assert (out[i, n:] == -7).all() and (grad_in[i, n:] == -7).all()
        _check_gated(name, x[i, :n], w[i], dy[i, :n], out[i, :n], (gi[i, :n], gw[i]), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("m,k,d,counts", [
    (1, 64, 96, [1, 0, 1]), (8, 130, 33, [8, 0, 3]), (16, 2048, 40, [16, 9, 0, 1]),
    (32, 72, 136, [0, 32, 17]), (32, 256, 40, [i % 33 for i in range(100)]),
    (20, 33, 130, [i % 21 for i in range(50)]), (100, 200, 72, [100, 0, 33, 64, 1, 96]),
    (128, 64, 300, [128, 5, 65] * 40), (129, 64, 40, [129, 0, 7])])
def test_experts_without_checkpoint(ga, name, m, k, d, counts, dtype):
    """The kernels for few rows: those that stream the weight, and the turned products."""
    x, w, _ = _operands(m, k, d, dtype, m + k, len(counts))
    for i, n in enumerate(counts):
        x[i, n:] = float("nan")
    out = torch.full((len(counts), m, d), -7.0, dtype=dtype, device="cuda")
    _ops(ga, name)[0](x, w, n_rows=torch.tensor(counts, dtype=torch.int32, device="cuda"), out=out)
    for i, n in enumerate(counts):
        assert (out[i, n:] == -7).all()
        _check_gated(name, x[i, :n], w[i], None, out[i, :n], None, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,d", [(1, 264, 9800), (16, 72, 10001), (32, 1030, 9728), (33, 520, 200),
                                   (64, 2000, 700), (128, 96, 9900), (100, 77, 333), (7, 8200, 24)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_few_rows(ga, m, k, d, pad, shift, dtype):
    x, w, _ = _operands(m, k, d, dtype, m + k)
    out = ga.linear_gelu_and_mul(_strided(x, pad, shift), _strided(w, pad, shift))
    _check_gated("gelu", x, w, None, out, None, dtype)


def _values(codes, scales):
    """What a LinearCheckpoint's codes [n, 2d] stand for, from the format's definition."""
    d, b = codes.shape[1] // 2, scales.shape[1] // 2
    step = 2.0 ** (scales.double() - 127)
    step = torch.where(scales == 255, torch.full_like(step, float("nan")), step)
    step = torch.cat([step[:, :b].repeat_interleave(32, 1)[:, :d],
                      step[:, b:].repeat_interleave(32, 1)[:, :d]], 1)
    return codes.double() * step, step


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,d", [(5, 64, 32), (40, 72, 33), (300, 100, 200)])
def test_checkpoint_values(ga, m, k, d, dtype):
    """Codes are the nearest multiples of the smallest step that holds their block."""
    x, w, _ = _operands(m, k, d, dtype, m)
    x[::3] *= 2.0 ** -9
    _, kept = ga.linear_silu_and_mul(x, w, keep=True)
    _, _, g, u, og, ou = R.forward("silu", x.double(), w.double(), dtype)
    ref, off = torch.cat([g, u], 1), torch.cat([og, ou], 1)
    values, step = _values(kept.codes, kept.scales)
    assert ((values - ref).abs() <= off + step / 2).all()
    top = torch.cat([R.block_top(g), R.block_top(u)], 1)
    worst = torch.cat([R.block_top(og), R.block_top(ou)], 1)
    assert ((top - worst) / step <= 32767.5).all() and ((top + worst) / step >= 16383.75).all()


def test_checkpoint_largest_code(ga):
    """Magnitudes just below a power of two, where the next step is taken once the largest code
    would round to 2^15: exact sums 2 - 2^-15 + t 2^-18 of three weights, alone in their blocks."""
    t = torch.arange(-16, 17, dtype=torch.float64)
    d = 32 * len(t)
    w = torch.zeros(2 * d, 8, dtype=torch.float64)
    rows = torch.arange(len(t)) * 32
    for base in (0, d):
        w[base + rows, 0] = 2 - 2.0 ** -7
        w[base + rows, 1] = 2.0 ** -7 - 2.0 ** -15
        w[base + rows, 2] = t * 2.0 ** -18
    exact = (w[:, 0] + w[:, 1] + w[:, 2])[rows]
    w = w.to(BF16)
    assert torch.equal(w.double().sum(1)[rows], exact)
    x = torch.ones(1, 8, dtype=BF16, device="cuda")
    out, kept = ga.linear_silu_and_mul(x, w.cuda(), keep=True)
    for part, base in ((0, 0), (1, d)):
        codes = kept.codes[0, base + rows.cuda()].cpu().double()
        scales = kept.scales[0].view(2, -1)[part].cpu().double()
        low = (exact * 2.0 ** 14).round() <= 32767          # ties to even: 32767.5 gives 32768
        assert torch.equal(scales, torch.where(low, 127.0 - 14, 127.0 - 13).double())
        assert torch.equal(codes, (exact / 2.0 ** (scales - 127)).round())
    dy = torch.ones(1, d, dtype=BF16, device="cuda")
    grads = ga.linear_silu_and_mul_backward(dy, x, w.cuda(), kept)
    _check_gated("silu", x, w.cuda(), dy, out, grads, BF16)


def test_gated_special_values(ga):
    """An infinity or a NaN reaches what it is multiplied into, and nothing else."""
    x, w, dy = _operands(70, 64, 40, BF16, 11)
    clean, kept = ga.linear_silu_and_mul(x, w, keep=True)
    grads = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    x[5, 3] = float("nan")
    x[66, 0] = float("inf")
    out, kept = ga.linear_silu_and_mul(x, w, keep=True)
    good = torch.ones(70, dtype=torch.bool, device="cuda")
    good[[5, 66]] = False
    assert torch.isnan(out[5]).all() and torch.equal(out[good], clean[good])
    gi, _ = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    assert torch.isnan(gi[5]).all() and torch.isnan(gi[66]).all()
    assert torch.equal(gi[good], grads[0][good])


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_wide_range(ga, dtype):
    """Rows of very different sizes keep their own precision: a scale for each 32 elements."""
    x, w, dy = _operands(96, 128, 100, dtype, 21)
    x *= (2.0 ** torch.linspace(-10, 6, 96, device="cuda")[:, None]).to(dtype)
    out, kept = ga.linear_gelu_and_mul(x, w, keep=True)
    _check_gated("gelu", x, w, dy, out, ga.linear_gelu_and_mul_backward(dy, x, w, kept), dtype)


@pytest.mark.parametrize("keep", [False, True])
def test_gated_long_sum(ga, keep):
    """A sum of 2^20 terms."""
    x, w, _ = _operands(3, 1 << 20, 8, BF16, 71)
    out = ga.linear_silu_and_mul(x, w, keep=keep)
    _check_gated("silu", x, w, None, out[0] if keep else out, None, BF16)


def test_gated_zero_sizes(ga):
    x, w, dy = _operands(0, 64, 32, BF16, 0)
    out, kept = ga.linear_silu_and_mul(x, w, keep=True)
    assert out.shape == (0, 32) and kept.codes.shape == (0, 64)
    gi, gw = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    assert gi.shape == (0, 64) and gw.shape == (64, 64) and (gw == 0).all()
    x, w, dy = _operands(4, 64, 32, BF16, 0, experts=0)
    assert ga.linear_silu_and_mul(x, w).shape == (0, 4, 32)


def test_gated_gradients_against_differences(ga):
    """sum(out * dy) in 64 bits from the kernels' forward output of moved fp16 operands would
    drown in rounding, so the differences are those of the 64-bit form, at the kernels' gradients."""
    x, w, dy = _operands(6, 16, 8, F16, 3)
    out, kept = ga.linear_gelu_and_mul(x, w, keep=True)
    gi, gw = ga.linear_gelu_and_mul_backward(dy, x, w, kept)

    def loss(x, w):
        h = x @ w.T
        a, _, _ = R.act("gelu", h[:, :8])
        return (a * h[:, 8:] * dy.double()).sum()

    for t, grad, which in ((x, gi, 0), (w, gw, 1)):
        for i in range(0, t.numel(), 7):
            at = [x.double(), w.double()]
            move = torch.zeros(t.numel(), dtype=torch.float64, device="cuda")
            move[i] = 1e-5
            move = move.view(t.shape)
            at[which] = at[which] + move
            up = loss(*at)
            at[which] = at[which] - 2 * move
            diff = (up - loss(*at)) / 2e-5
            # fp16 roundings of the factors (2^-11 each, up to 96 terms of about unit size)
            assert abs(grad.reshape(-1)[i].item() - diff.item()) <= 96 * 2.0 ** -11 + 2.0 ** -11 * abs(diff)


# ------------------------------------------------------------- cross entropy

def _tokens(t, k, v, dtype, seed, live=1.0):
    x = _randn(t, k, seed=seed).to(dtype)
    w = _randn(v, k, seed=seed + 1, scale=2 * k ** -0.5).to(dtype)
    goal = torch.randint(v, (t,), generator=_gen(seed + 2), device="cuda")
    if live < 1:
        dead = torch.rand(t, generator=_gen(seed + 3), device="cuda") >= live
        goal = torch.where(dead, torch.full_like(goal, -100), goal)
    gl = (0.25 + torch.rand(t, generator=_gen(seed + 4), device="cuda"))
    return x, w, goal, gl


def _check_entropy(x, w, goal, gl, kept, grads, dtype):
    live = (goal >= 0) & (goal < len(w))
    assert (kept.loss[~live] == 0).all() and (kept.lse[~live] == 0).all()
    xl, wl, at = x[live].double(), w.double(), goal[live].long()
    if live.any():
        loss, bl, lse, bs, _, _ = R.entropy(xl, wl, at)
        R.check(kept.loss[live], loss, bl, "loss")
        R.check(kept.lse[live], lse, bs, "lse")
    gi, gw = grads
    assert (gi[~live] == 0).all()
    (ri, bi), (rw, bw) = R.entropy_backward(gl[live].double(), xl, wl, at, dtype)
    R.check(gi[live], ri, bi, "grad_in")
    R.check(gw, rw, bw, "grad_weight")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("live", [1.0, 0.4])
@pytest.mark.parametrize("t,k,v", ENTROPY)
def test_entropy(ga, t, k, v, live, dtype):
    x, w, goal, gl = _tokens(t, k, v, dtype, t + k + v, live)
    kept = ga.linear_cross_entropy(x, w, goal)
    _check_entropy(x, w, goal, gl, kept, ga.linear_cross_entropy_backward(gl, x, w, goal, kept), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_entropy_dead_tokens(ga, dtype):
    """What lies in a dead token's row, or comes to it as a gradient, has no effect."""
    x, w, goal, gl = _tokens(300, 72, 500, dtype, 9, 0.5)
    dead = goal < 0
    goal[dead.nonzero()[::2, 0]] = 500          # past the vocabulary, as good as -100
    x[dead] = float("nan")
    gl[dead] = float("inf")
    kept = ga.linear_cross_entropy(x, w, goal.int())
    grads = ga.linear_cross_entropy_backward(gl, x, w, goal.int(), kept)
    _check_entropy(x, w, goal, gl, kept, grads, dtype)
    goal.fill_(-1)
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    assert not any(t.any() for t in (kept.loss, kept.lse, gi, gw))


@pytest.mark.parametrize("k", [40, 1100])
def test_entropy_many_tokens(ga, k):
    """More tokens than all SMs number in one turn, and rows of more than one piece."""
    x, w, goal, gl = _tokens(170001 if k < 100 else 5000, k, 50, BF16, k, 0.6)
    kept = ga.linear_cross_entropy(x, w, goal)
    grads = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    _check_entropy(x, w, goal, gl, kept, grads, BF16)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 5), (0, 1)])
def test_entropy_strides(ga, pad, shift):
    x, w, goal, gl = _tokens(130, 80, 600, BF16, 4, 0.9)
    kept = ga.linear_cross_entropy(x, w, goal)
    grads = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    xs, ws = _strided(x, pad, shift), _strided(w, pad, shift)
    again = ga.linear_cross_entropy(xs, ws, goal)
    assert torch.equal(again.loss, kept.loss)
    for a, b in zip(ga.linear_cross_entropy_backward(gl, xs, ws, goal, again), grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_entropy_far_logits(ga, dtype):
    """Logits of hundreds: the row's own maximum is taken out first."""
    x, w, goal, gl = _tokens(64, 64, 700, dtype, 6)
    x *= 40
    kept = ga.linear_cross_entropy(x, w, goal)
    _check_entropy(x, w, goal, gl, kept, ga.linear_cross_entropy_backward(gl, x, w, goal, kept), dtype)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -30, 2.0 ** 20])
def test_entropy_gradient_scales(ga, scale):
    x, w, goal, gl = _tokens(90, 64, 300, BF16, 8)
    gl = gl * scale
    gl[::3] *= 1e-3
    kept = ga.linear_cross_entropy(x, w, goal)
    _check_entropy(x, w, goal, gl, kept, ga.linear_cross_entropy_backward(gl, x, w, goal, kept), BF16)


def test_entropy_zero_tokens(ga):
    x, w, goal, gl = _tokens(0, 64, 300, BF16, 8)
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    assert kept.loss.shape == (0,) and gi.shape == (0, 64) and (gw == 0).all()


def test_entropy_gradients_against_differences(ga):
    """The kernels' gradients against differences of the 64-bit form."""
    x, w, goal, gl = _tokens(7, 16, 40, F16, 12, 0.8)
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    live = goal >= 0
    loss = lambda x, w: (R.entropy(x[live], w, goal[live])[0] * gl[live].double()).sum()  # noqa: E731
    (_, bounds_in), (_, bounds_w) = R.entropy_backward(gl[live].double(), x[live].double(), w.double(),
                                                       goal[live], F16)
    full = torch.zeros_like(x, dtype=torch.float64)
    full[live] = bounds_in
    for t, grad, bound, which in ((x, gi, full, 0), (w, gw, bounds_w, 1)):
        for i in range(0, t.numel(), 13):
            move = torch.zeros(t.numel(), dtype=torch.float64, device="cuda")
            move[i] = 1e-5
            at = [x.double(), w.double()]
            up, down = list(at), list(at)
            up[which] = at[which] + move.view(t.shape)
            down[which] = at[which] - move.view(t.shape)
            diff = (loss(*up) - loss(*down)) / 2e-5
            # the differences' own error: a third derivative times 1e-10, and cancellation
            assert abs(grad.reshape(-1)[i].item() - diff.item()) <= bound.reshape(-1)[i].item() + 1e-6


# ------------------------------------------------------------------ many sizes

def test_random_sizes(ga):
    import random
    rng = random.Random(20)
    for i in range(40):
        dtype, name = rng.choice(DTYPES), rng.choice(["silu", "gelu"])
        m, k, d = (int(2 ** rng.uniform(0, hi)) for hi in (9.5, 9, 9))
        if rng.random() < 0.5:
            x, w, dy = _operands(m, k, d, dtype, i)
            out, kept = _ops(ga, name)[0](x, w, keep=True)
            _check_gated(name, x, w, dy, out, _ops(ga, name)[1](dy, x, w, kept), dtype)
            _check_gated(name, x, w, None, _ops(ga, name)[0](x, w), None, dtype)
        else:
            v = int(2 ** rng.uniform(0, 13))
            x, w, goal, gl = _tokens(m, k, v, dtype, i, rng.choice([1.0, 0.7]))
            kept = ga.linear_cross_entropy(x, w, goal)
            _check_entropy(x, w, goal, gl, kept,
                           ga.linear_cross_entropy_backward(gl, x, w, goal, kept), dtype)


def test_offsets_past_32_bits_gated(ga):
    """Outputs, codes and gradients of more than 2^31 elements."""
    m, k, d = 70000, 64, 32768
    x, w, _ = _operands(m, k, d, BF16, 81)
    out, kept = ga.linear_silu_and_mul(x, w, keep=True)
    dy = torch.empty(m, d, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 255, 32767, 65535, 65536, 69999], device="cuda")
    dy.zero_()
    dy[rows] = _randn(len(rows), d, seed=82).to(BF16)
    _check_gated("silu", x[rows], w, None, out[rows], None, BF16)
    gi, gw = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    # the other rows add nothing
    (ri, bi), (rw, bw) = R.backward("silu", dy[rows].double(), x[rows].double(), w.double(), BF16)
    R.check(gi[rows], ri, bi, "grad_in")
    R.check(gw, rw, bw, "grad_weight")


def test_offsets_past_32_bits_entropy(ga):
    """A weight of more than 2^31 elements."""
    t, k, v = 40, 8200, 270000
    w = torch.empty(v, k, dtype=BF16, device="cuda")
    for i in range(0, v, 30000):
        w[i:i + 30000] = _randn(30000, k, seed=i, scale=2 * k ** -0.5).to(BF16)
    x = _randn(t, k, seed=1).to(BF16)
    goal = torch.randint(v, (t,), generator=_gen(2), device="cuda")
    goal[0], goal[1] = v - 1, 0
    gl = torch.rand(t, generator=_gen(3), device="cuda")
    kept = ga.linear_cross_entropy(x, w, goal)
    gi, gw = ga.linear_cross_entropy_backward(gl, x, w, goal, kept)
    # the logits in 64 bits, in parts; then a part of the vocabulary's gradient
    logits = torch.cat([x.double() @ w[i:i + 30000].double().T for i in range(0, v, 30000)], 1)
    lse = torch.logsumexp(logits, 1)
    at = logits.gather(1, goal[:, None])[:, 0]
    off = R.acc(k) * (x.double().abs().sum(1) * w.abs().max().item())
    assert ((kept.lse - lse).abs() <= off + 1e-4).all() and ((kept.loss - (lse - at)).abs() <= 2 * off + 1e-4).all()
    y = torch.exp(logits - lse[:, None])
    y[torch.arange(t, device="cuda"), goal] -= 1
    y *= gl.double()[:, None]
    for part in (slice(0, 300), slice(261000, 262500), slice(v - 300, v)):
        ref = y[:, part].T @ x.double()
        # half a step of y and of the result, and y's own error: off of exp's argument, at most
        loose = (y[:, part].abs() * (2.0 ** -8 + 3 * off[:, None] + 1e-4)).T @ x.double().abs()
        R.check(gw[part], ref, loose + R.half_step(ref, BF16) + 1e-30, "grad_weight")
    ref = sum(y[:, i:i + 30000] @ w[i:i + 30000].double() for i in range(0, v, 30000))
    # row by row in norm: y's roundings are independent of each other and of the weight
    assert ((gi.double() - ref).norm(dim=1) <= 2 * 2.0 ** -8 * ref.norm(dim=1)).all()


# ------------------------------------------------------- streams, graphs, order

def test_runs_together(ga):
    """A gated block, its loss and both gradients in a row, on another stream than the default
    one, twice; captured into a graph and replayed with other inputs."""
    x, w, _ = _operands(200, 128, 96, BF16, 31)
    head = _randn(1000, 96, seed=32, scale=0.1).to(BF16)
    goal = torch.randint(1000, (200,), generator=_gen(33), device="cuda")
    gl = torch.full((200,), 1 / 200, device="cuda")

    def step():
        y, kept = ga.linear_silu_and_mul(x, w, keep=True)
        ce = ga.linear_cross_entropy(y, head, goal)
        gy, ghead = ga.linear_cross_entropy_backward(gl, y, head, goal, ce)
        return (y, ce.loss, ghead) + ga.linear_silu_and_mul_backward(gy, x, w, kept)

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    # the whole against autograd in 64 bits: by norm, as roundings of the steps between add up
    xd, wd, hd = (t.double().requires_grad_() for t in (x, w, head))
    h = xd @ wd.T
    yd = torch.nn.functional.silu(h[:, :96]) * h[:, 96:]
    torch.nn.functional.cross_entropy(yd @ hd.T, goal).backward()
    for got, ref in ((want[2], hd.grad), (want[3], xd.grad), (want[4], wd.grad)):
        # three roundings of half a step each, on the way to a gradient and in it
        assert (got.double() - ref).norm() <= 3 * 2.0 ** -8 * ref.norm()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x2, _, _ = _operands(200, 128, 96, BF16, 77)
    old = x.clone()
    x.copy_(x2)
    other = step()
    x.copy_(old)
    for source, result in ((old, want), (x2, other), (old, want)):
        x.copy_(source)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, result))


def test_block_of_experts(ga):
    """examples/train_mlp_block.py with its experts' products fused: gradients against autograd of
    the same block in 64 bits, and a few training steps."""
    import importlib
    example = importlib.import_module("examples.train_mlp_block")
    s = example.Shape(tokens=96, width=64, d=48, experts=4, k=2)
    block = example.Block(s, "fused", seed=3)
    x = _randn(s.tokens, s.width, seed=5).to(BF16)
    grad_y = _randn(s.tokens, s.width, seed=6).to(BF16)
    y, loss, saved = block.forward(x)
    grad_x, grads = block.backward(grad_y, torch.full((1,), 2.0, device="cuda"), saved)

    p = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xr, ids = x.double().requires_grad_(), saved[5]
    normed = torch.nn.functional.layer_norm(xr, (s.width,), p["norm_weight"], p["norm_bias"], 1e-5)
    full = torch.softmax(normed @ p["router"], 1)
    ref = xr
    for j in range(s.k):
        e = ids[:, j]
        h = torch.einsum("tw,tdw->td", normed, p["up"][e])
        a = torch.nn.functional.silu(h[:, :s.d]) * h[:, s.d:]
        ref = ref + full.gather(1, e[:, None]) * torch.einsum("td,tdw->tw", a, p["down"][e])
    counts = torch.bincount(ids.reshape(-1), minlength=s.experts).double()
    balance = s.coef * s.experts * (counts / (s.tokens * s.k) * full.mean(0)).sum()
    ((ref * grad_y.double()).sum() + 2 * balance).backward()

    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    # eight bf16 roundings of half a step lie on the way of a gradient through the block (its input,
    # the products and their operands), in norm at most 8 x 2^-8 with none of them cancelled
    assert off(y, ref.detach()) < 8 * 2.0 ** -8 and off(loss, balance.detach().view(1)) < 0.01
    assert off(grad_x, xr.grad) < 8 * 2.0 ** -8
    for name, value in p.items():
        assert off(grads[name], value.grad) < 8 * 2.0 ** -8, name
    assert len(example.train(steps=3, activation="fused", shape=s)) == 3


def test_many_passes_in_a_row(ga):
    """Kernels of one and two CTAs per SM pair behind each other without a pause, some of them on
    a part of the SMs: 1500 launches of products."""
    x, w, dy = _operands(1001, 1101, 2731, F16, 61)
    for _ in range(500):
        out, kept = ga.linear_silu_and_mul(x, w, keep=True)
        grads = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    torch.cuda.synchronize()
    _check_gated("silu", x, w, dy, out, grads, F16)


def test_two_streams_at_once(ga):
    """Calls that overlap on the GPU have workspaces of their own."""
    x, w, dy = _operands(500, 257, 300, BF16, 41)
    want, kept = ga.linear_silu_and_mul(x, w, keep=True)
    grads = ga.linear_silu_and_mul_backward(dy, x, w, kept)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            out, k = ga.linear_silu_and_mul(x, w, keep=True, stream=s)
            got.append((out, *ga.linear_silu_and_mul_backward(dy, x, w, k, stream=s)))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, (want, *grads)))


def test_threads(ga):
    """Calls from three threads at once, each on a stream of its own."""
    import threading
    x, w, dy = _operands(200, 130, 96, BF16, 65)
    goal = torch.randint(192, (200,), generator=_gen(66), device="cuda")
    gl = torch.ones(200, device="cuda")

    def work():
        out, kept = ga.linear_silu_and_mul(x, w, keep=True)
        ce = ga.linear_cross_entropy(x, w, goal)
        return (out, *ga.linear_silu_and_mul_backward(dy, x, w, kept), ce.loss,
                *ga.linear_cross_entropy_backward(gl, x, w, goal, ce))

    want, got = work(), []
    torch.cuda.synchronize()

    def run():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                result = work()
        stream.synchronize()
        got.append(result)

    threads = [threading.Thread(target=run) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 3
    for result in got:
        assert all(torch.equal(a, b) for a, b in zip(result, want))


def test_two_graphs(ga):
    """Two captured graphs, replayed in turn and on two streams at once."""
    sets = [_operands(300, 200, 130, BF16, 90 + i) for i in range(2)]
    goals = [torch.randint(200, (300,), generator=_gen(i), device="cuda") for i in range(2)]
    gl = torch.full((300,), 1 / 300, device="cuda")

    def work(i):
        x, w, dy = sets[i]
        out, kept = ga.linear_gelu_and_mul(x, w, keep=True)
        ce = ga.linear_cross_entropy(x, w, goals[i])
        return (out, *ga.linear_gelu_and_mul_backward(dy, x, w, kept), ce.loss,
                *ga.linear_cross_entropy_backward(gl, x, w, goals[i], ce))

    want = [work(0), work(1)]
    torch.cuda.synchronize()
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            held.append(work(i))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(held, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_autograd_function(ga):
    """The two passes in a torch.autograd.Function."""
    class Up(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            out, kept = ga.linear_silu_and_mul(x, w, keep=True)
            ctx.save_for_backward(x, w, *kept)
            return out

        @staticmethod
        def backward(ctx, grad):
            x, w, *kept = ctx.saved_tensors
            return ga.linear_silu_and_mul_backward(grad.contiguous(), x, w, ga.LinearCheckpoint(*kept))

    x, w, _ = _operands(50, 64, 32, BF16, 51)
    x.requires_grad_()
    w.requires_grad_()
    Up.apply(x, w).sum().backward()
    ones = torch.ones(50, 32, dtype=torch.float64, device="cuda")
    want = R.backward("silu", ones, x.detach().double(), w.detach().double(), BF16)
    for got, (ref, bound) in zip((x.grad, w.grad), want):
        R.check(got, ref, bound, "gradient")


# ------------------------------------------------------------------- refusals

def test_refusals(ga):
    x, w, dy = _operands(4, 16, 8, BF16, 1)
    out, kept = ga.linear_silu_and_mul(x, w, keep=True)
    f, b = ga.linear_silu_and_mul, ga.linear_silu_and_mul_backward
    with pytest.raises(TypeError):
        f(x.float(), w.float())
    for bad in (lambda: f(x, w.half()), lambda: f(x, w[:15]), lambda: f(x, w[:, :8]),
                lambda: f(x.T, w), lambda: f(x[None], w), lambda: f(x.cpu(), w),
                lambda: f(x.cpu().pin_memory(), w), lambda: f(x, w, out=out[:, :4]),
                lambda: f(x, w, n_rows=torch.ones(1, device="cuda")),
                lambda: f(x, w, n_rows=torch.ones(2, dtype=torch.int32, device="cuda")),
                lambda: f(x, w, n_rows=torch.ones(1, dtype=torch.int32)),
                lambda: b(dy[:, :4], x, w, kept), lambda: b(dy.half(), x, w, kept),
                lambda: b(dy, x, w, ga.LinearCheckpoint(kept.codes[:2], kept.scales)),
                lambda: b(torch.zeros(1, 1, dtype=BF16, device="cuda").expand(4, 8), x, w, kept)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        b(dy, x, w, kept.codes)
    with pytest.raises(ga.GatedActError):       # every row the same memory
        f(x[:1].expand(4, 16), w)
    with pytest.raises(ga.GatedActError):       # the output over the input
        f(x, w, out=x.view(-1)[:32].view(4, 8))
    e = ga.linear_cross_entropy
    goal = torch.zeros(4, dtype=torch.int64, device="cuda")
    ce = e(x, w, goal)
    for bad in (lambda: e(x, w.half(), goal), lambda: e(x, w, goal[:3]), lambda: e(x, w[:, :8], goal),
                lambda: e(x, w, goal.cpu()), lambda: e(x[None], w[None], goal),
                lambda: ga.linear_cross_entropy_backward(ce.loss.double(), x, w, goal, ce),
                lambda: ga.linear_cross_entropy_backward(ce.loss[:1].expand(4), x, w, goal, ce)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        e(x, w, goal.float())
