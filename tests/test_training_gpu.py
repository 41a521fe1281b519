"""The training operators on the GPU against their 64-bit forms (tests/training_ref.py, which
derives the bounds): 8-bit checkpoints and the backward passes that read them, layer norm, the
balance loss."""
import ctypes

import pytest
import torch

import workloads as W
from tests import training_ref as R
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF16, F16, F32]
# rows x width: one element, below and above a block, rows that start unaligned, vector widths
# with and without a ragged last block, an expert's width, several vectors per thread, wider
# than a row that one CTA holds
SHAPES = [(1, 1), (3, 7), (5, 32), (2, 33), (4, 40), (3, 96), (64, 257), (33, 768), (7, 4099),
          (5, 8192), (2, 16392), (2, 32768), (1, 40000), (3, 1500), (2, 8001), (2, 16001),
          (1, 32761), (1, 40001)]


@pytest.fixture(scope="module")
def ga():
    return require_gpu()


def _randn(*shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return scale * torch.randn(shape, generator=g)


def _gated(m, d, dtype, seed, pad=0, shift=0):
    """[M, 2d + pad] rows: gates with a mean and a scale of their own and some outliers; the
    padding is NaN, and `shift` elements of it come before the first row."""
    gate = _randn(m, d, seed=seed) * (0.5 + _randn(m, 1, seed=seed + 1).abs()) \
        + 0.5 * _randn(m, 1, seed=seed + 2)
    gate = torch.where(_randn(m, d, seed=seed + 3) > 2.3, 4 * gate, gate)
    buf = torch.full((shift + m * (2 * d + pad),), float("nan"))
    x = buf[shift:].view(m, 2 * d + pad)
    x[:, :2 * d] = torch.cat([gate, _randn(m, d, seed=seed + 4)], 1)
    return buf.to(dtype).cuda()[shift:].view(m, 2 * d + pad)


def _ops(ga, name):
    return {"silu": (ga.silu_and_mul_checkpoint, ga.silu_and_mul_backward),
            "gelu": (ga.gelu_and_mul_checkpoint, ga.gelu_and_mul_backward)}[name]


def _strided(x, pad, shift):
    m, n = x.shape
    buf = torch.full((shift + m * (n + pad),), float("nan"), dtype=x.dtype)
    view = buf[shift:].view(m, n + pad)
    view[:, :n] = x
    return buf.cuda()[shift:].view(m, n + pad)[:, :n]


# --------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_checkpoint_step(ga, name, m, d, dtype):
    x = _gated(m, d, dtype, 10 * d + m)
    forward, backward = _ops(ga, name)
    out, kept = forward(x)
    xr = x.double().cpu()
    a, _, _, grow = R.act(name, xr[:, :d])
    ref = a * xr[:, d:]
    R.check(out, ref, ref.abs() * grow, dtype, "out")
    gate, up = R.encode(xr[:, :d]), R.encode(xr[:, d:])
    assert torch.equal(kept.codes.cpu(), torch.cat([gate[0], up[0]], 1))
    assert torch.equal(kept.scales.cpu(), torch.cat([gate[1], up[1]], 1))
    v = R.values(kept.codes, kept.scales)
    for t in (BF16, F32):
        assert torch.equal(ga.checkpoint_values(kept, t).double().cpu(), v)
    dy = _randn(m, d, seed=d).to(dtype)
    grad, again = backward(dy.cuda(), kept, recompute=True)
    want = R.act_backward(name, v, dy.double())
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(again, *want["out"], dtype, "recomputed out")
    only = backward(dy.cuda(), kept)
    assert torch.equal(only, grad)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(3, 0), (8, 0), (0, 1), (40, 8)])
@pytest.mark.parametrize("d", [40, 256])
def test_checkpoint_layouts_give_the_same_bits(ga, d, pad, shift, dtype):
    # rows of a wider buffer, rows that start off a 16-byte boundary: same results as contiguous
    m = 9
    x = _gated(m, d, dtype, 5, pad, shift)
    flat = x[:, :2 * d].contiguous()
    dy = _randn(m, d, seed=6).to(dtype)
    for name in ("silu", "gelu"):
        forward, backward = _ops(ga, name)
        (o1, k1), (o2, k2) = forward(x, d=d), forward(flat)
        assert torch.equal(o1, o2) and torch.equal(k1.codes, k2.codes)
        assert torch.equal(k1.scales, k2.scales)
        g1 = backward(_strided(dy, pad, shift), k1)
        assert torch.equal(g1, backward(dy.cuda(), k2))
    (o1, k1), (o2, k2) = (ga.gelu_and_mul_sparse_checkpoint(v, 0.5, d=d) for v in (x, flat))
    xr = flat.double().cpu()
    _check_sparse_forward(xr, d, 0.5, dtype, o1, k1)
    _check_sparse_forward(xr, d, 0.5, dtype, o2, k2)
    want = R.sparse_backward(R.values(k1.codes, k1.scales), dy.double(), k1.std.double().cpu(), 0.5)
    for g in (_strided(dy, pad, shift), dy.cuda()):
        R.check(ga.gelu_and_mul_sparse_backward(g, k1, 0.5), *want["grad"], dtype, "grad")


@pytest.mark.parametrize("n", [-2, 0, 1, 31, 64, 100])
@pytest.mark.parametrize("d", [64, 37])
def test_checkpoint_live_rows(ga, d, n):
    m = 64
    x = _gated(m, d, BF16, 7)
    lib, live = ga.load_library(), min(max(n, 0), m)
    nr = torch.tensor([n], dtype=torch.int32, device="cuda")
    full, kfull = ga.silu_and_mul_checkpoint(x)
    out = torch.full((m, d), 7.0, dtype=BF16, device="cuda")
    codes = torch.full((m, 2 * d), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((m, 2 * -(-d // 32)), 33, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert lib.silu_and_mul_checkpoint(out.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                       x.data_ptr(), m, d, 2 * d, ga.BF16, nr.data_ptr(), s) == 0
    grad = torch.full((m, 2 * d), 7.0, dtype=BF16, device="cuda")
    dy = _randn(m, d, seed=8).to(BF16).cuda()
    assert lib.silu_and_mul_backward(grad.data_ptr(), None, dy.data_ptr(), kfull.codes.data_ptr(),
                                     kfull.scales.data_ptr(), m, d, d, ga.BF16, nr.data_ptr(),
                                     s) == 0
    for got, want, rest in ((out, full, 7.0), (codes, kfull.codes, 99), (scales, kfull.scales, 33),
                            (grad, ga.silu_and_mul_backward(dy, kfull), 7.0)):
        assert torch.equal(got[:live], want[:live]) and (got[live:] == rest).all()


def test_checkpoint_special_values(ga):
    # zeros, subnormals, the largest values, infinities and NaN: codes by the definition, NaN
    # kept inside its block
    d = 96
    x = _randn(6, 2 * d, seed=9)
    x[0, :32] = 0
    x[1, :64] *= 1e-38
    x[1, 64:96] = 1.4e-45
    x[2, 32:64] = 3.4e38
    x[3, 40] = float("inf")
    x[4, 70] = float("nan")
    x[5, 100] = -float("inf")
    for dtype in (F32, BF16):
        xd = x.to(dtype).cuda()
        _, kept = ga.silu_and_mul_checkpoint(xd)
        xr = xd.double().cpu()
        gate, up = R.encode(xr[:, :d]), R.encode(xr[:, d:])
        assert torch.equal(kept.codes.cpu(), torch.cat([gate[0], up[0]], 1))
        assert torch.equal(kept.scales.cpu(), torch.cat([gate[1], up[1]], 1))
        v = R.values(kept.codes, kept.scales)
        assert torch.equal(torch.isnan(ga.checkpoint_values(kept)).cpu(), torch.isnan(v))
        grad = ga.silu_and_mul_backward(torch.ones(6, d, dtype=dtype, device="cuda"), kept)
        bad = torch.isnan(v[:, :d]) | torch.isnan(v[:, d:])
        got = torch.isnan(grad).cpu()
        assert torch.equal(got[:, :d], bad) and torch.equal(got[:, d:], torch.isnan(v[:, :d]))


def test_activation_slope_far_out(ga):
    # gates up to the type's range: the slope tends to 0 and 1, with no inf * 0 on the way
    g = torch.tensor([[-3e38, -1e20, -200.0, -30.0, 30.0, 200.0, 1e20, 3e38]]).repeat(1, 4)
    for i in range(8):     # each value alone in its block, so that it is held exactly enough
        gate = g[:, i:i + 1].expand(1, 32).contiguous()
        x = torch.cat([gate, torch.ones(1, 32)], 1).cuda()
        for name in ("silu", "gelu"):
            forward, backward = _ops(ga, name)
            grad = backward(torch.ones(1, 32, device="cuda"), forward(x)[1])[0, :32]
            assert torch.allclose(grad, (g[0, i] > 0).float().cuda().expand(32), atol=1e-9), name


def _check_sparse_forward(xr, d, z, dtype, out, kept):
    mean, std, delta = R.sparse_stats(xr, d, z)
    # the fp32 cutoff is off by at most 2^-20 of what it is made of
    off = 2.0 ** -20 * (xr[:, :d].abs().mean(1, keepdim=True) + mean.abs() + (1 + abs(z)) * std)
    R.check(kept.std, std[:, 0], (std + xr[:, :d].abs().mean(1, keepdim=True))[:, 0], F32, "std")
    s = delta.clamp(min=0)
    a, _, _, grow = R.act("gelu", s)
    ref = a * xr[:, d:]
    R.check(out, ref, ref.abs() * grow + 2.0 ** 18 * off * xr[:, d:].abs() * 1.2, dtype, "out")
    codes, scales = kept.codes.cpu(), kept.scales.cpu()
    B = scales.shape[1] // 2
    step = R.steps(scales[:, :B], d)
    v = codes[:, :d].double() * step
    sure = delta.abs() > off
    assert torch.equal((codes[:, :d] > 0)[sure], (delta > 0)[sure])
    raised = (delta > -off) & (delta < step / 2 + off)           # a positive value's code is >= 1
    assert ((v - delta).abs() <= torch.where(raised, step, step / 2) + off).all()
    top = R.blocks(v.abs()).amax(2)
    full = scales[:, :B] > 0
    assert (R.blocks(codes[:, :d].double().abs()).amax(2)[full] >= 63).all() and top.isfinite().all()
    up = R.encode(xr[:, d:])
    assert torch.equal(codes[:, d:], up[0]) and torch.equal(scales[:, B:], up[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("z", [0.0, W.Z95, -0.5])
@pytest.mark.parametrize("m,d", SHAPES)
def test_sparse_step(ga, m, d, z, dtype):
    x = _gated(m, d, dtype, 20 * d + m)
    out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z)
    xr = x.double().cpu()
    _check_sparse_forward(xr, d, z, dtype, out, kept)
    v = R.values(kept.codes, kept.scales)
    dy = _randn(m, d, seed=d + 1).to(dtype)
    want = R.sparse_backward(v, dy.double(), kept.std.double().cpu(), z)
    grad, again = ga.gelu_and_mul_sparse_backward(dy.cuda(), kept, z, recompute=True)
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(again, *want["out"], dtype, "recomputed out")
    assert torch.equal(ga.gelu_and_mul_sparse_backward(dy.cuda(), kept, z), grad)


# more rows of each width than two per CTA of the GPU, and not a multiple of its CTAs
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,d", [(2437, 1032), (2501, 2048), (1219, 2056), (1243, 4096),
                                 (613, 4104), (611, 8192), (307, 8200), (311, 16384)])
def test_sparse_long_batches(ga, m, d, dtype):
    x = _gated(m, d, dtype, d + m, pad=8)[:, :2 * d]
    out, kept = ga.gelu_and_mul_sparse_checkpoint(x, W.Z95)
    _check_sparse_forward(x.double().cpu(), d, W.Z95, dtype, out, kept)
    dy = _randn(m, d, seed=m).to(dtype)
    want = R.sparse_backward(R.values(kept.codes, kept.scales), dy.double(),
                             kept.std.double().cpu(), W.Z95)
    grad, again = ga.gelu_and_mul_sparse_backward(_strided(dy, 8, 0), kept, W.Z95, recompute=True)
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(again, *want["out"], dtype, "recomputed out")
    # a row's results are its own, whichever CTA takes it
    for rows in (slice(0, 1), slice(m - 1, m), slice(m // 2, m // 2 + 1)):
        part = type(kept)(*(t[rows] for t in kept))
        alone = ga.gelu_and_mul_sparse_backward(dy[rows].cuda(), part, W.Z95)
        R.check(alone, *(t[rows] for t in want["grad"]), dtype, "grad of a row")


@pytest.mark.parametrize("d", [64, 45, 2048])
def test_sparse_constant_and_masked_rows(ga, d):
    # constant gates (std = 0): nothing passes, gradients are 0; gradients that are not finite
    # where the mask is 0 stay out of the row's sum
    x = torch.cat([torch.full((3, d), 0.75), _randn(3, d, seed=1)], 1).to(BF16).cuda()
    for z in (0.0, W.Z95, -1.0):
        out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z)
        assert (out == 0).all() and (kept.std == 0).all() and (kept.codes[:, :d] <= 0).all()
        grad = ga.gelu_and_mul_sparse_backward(torch.ones(3, d, dtype=BF16, device="cuda"), kept, z)
        assert (grad == 0).all()
    x = _gated(2, d, F32, 3)
    _, kept = ga.gelu_and_mul_sparse_checkpoint(x, 1.0)
    dy = _randn(2, d, seed=2).cuda()
    clean = ga.gelu_and_mul_sparse_backward(dy, kept, 1.0)
    off = kept.codes[0, :d] <= 0
    dy[0, off] = float("inf")
    dy[0, off.nonzero()[0]] = float("nan")
    assert torch.equal(ga.gelu_and_mul_sparse_backward(dy, kept, 1.0)[:, :d], clean[:, :d])


def test_sparse_nan_row_stays_in_its_row(ga):
    d = 512
    x = _gated(3, d, BF16, 4)
    x[1, 5] = float("nan")
    out, kept = ga.gelu_and_mul_sparse_checkpoint(x, 1.0)
    grad = ga.gelu_and_mul_sparse_backward(torch.ones(3, d, dtype=BF16, device="cuda"), kept, 1.0)
    for t in (out, grad):
        bad = torch.isnan(t).any(1).tolist()
        assert bad == [False, True, False]
    assert torch.isnan(out[1]).all() and torch.isnan(grad[1]).all()
    assert (kept.codes[1, :d] == 0).all() and (kept.scales[1, :d // 32] == 255).all()


@pytest.mark.parametrize("name", ["silu", "gelu", "sparse"])
def test_gradient_against_differences_of_the_kernels(ga, name):
    # values that the checkpoint holds exactly; fp32 differences of the library's own forward pass
    m, d, z, h = 4, 64, 0.5, 2.0 ** -6
    q = torch.randint(-127, 128, (m, 2 * d), generator=torch.Generator().manual_seed(3))
    q[:, ::32] = 127
    x = (q.float() / 64).cuda()
    dy = _randn(m, d, seed=5).cuda()

    def f(x):
        if name == "sparse":
            return ga.gelu_and_mul_sparse(x, z)
        return _ops(ga, name)[0](x)[0]

    if name == "sparse":
        # held to the rounding of gate - cutoff: half a step of its slope's change, z's term
        kept = ga.gelu_and_mul_sparse_checkpoint(x, z)[1]
        grad, tol = ga.gelu_and_mul_sparse_backward(dy, kept, z), 0.06
    else:
        kept = _ops(ga, name)[0](x)[1]
        grad, tol = _ops(ga, name)[1](dy, kept), 2e-3
    torch.manual_seed(0)
    for c in (0, 5, 33, d, d + 7, 2 * d - 1):
        e = torch.zeros_like(x)
        e[:, c] = h
        diff = ((f(x + e) - f(x - e)) * dy).double().sum(1) / (2 * h)
        if name == "sparse" and c < d:       # away from the kink the difference is of one side
            delta = R.sparse_stats(x.double().cpu(), d, z)[2]
            far = (delta.abs() > 3 * h).all(1) | (delta[:, c].abs() > 3 * h)
            diff, got = diff[far.cuda()], grad[far.cuda(), c].double()
        else:
            got = grad[:, c].double()
        assert ((diff - got).abs() <= tol * (1 + dy.abs().amax().double() * 2)).all(), c


# ---------------------------------------------------------------- layer norm

def _norm_case(t, d, dtype, wtype, seed, bias=True):
    x = (_randn(t, d, seed=seed) * (0.5 + _randn(t, 1, seed=seed + 1).abs())
         + _randn(t, 1, seed=seed + 2)).to(dtype)
    w = (1 + 0.2 * _randn(d, seed=seed + 3)).to(wtype)
    b = (0.3 * _randn(d, seed=seed + 4)).to(wtype) if bias else None
    return x, w, b, _randn(t, d, seed=seed + 5).to(dtype)


# and many rows: aligned and off a boundary, through every number of rows per CTA, and rows
# that a cluster shares
NORM_SHAPES = SHAPES + [(700, 2048), (1000, 40), (320, 8192), (300, 1), (5000, 301), (3000, 520),
                        (1300, 2047), (1000, 4099), (650, 1036), (170, 20000), (170, 12345)]


def _check_norm(ga, x, w, b, dy, dtype, eps=1e-5, xd=None, dyd=None):
    t, d = x.shape
    xd = x.cuda() if xd is None else xd
    dyd = dy.cuda() if dyd is None else dyd
    wd, bd = w.cuda(), b.cuda() if b is not None else None
    out, mean, rstd = ga.layer_norm(xd, wd, bd, eps)
    # the kernel takes eps in fp32
    eps32 = float(torch.tensor(eps, dtype=F32))
    want = R.layer_norm(x.double(), w.double(), b.double() if b is not None else None, eps32)
    R.check(out, *want["out"], dtype, "out")
    R.check(mean, *want["mean"], F32, "mean")
    R.check(rstd, *want["rstd"], F32, "rstd")
    grad, gw, gb = ga.layer_norm_backward(dyd, xd, wd, mean, rstd, bias=b is not None)
    want = R.layer_norm_backward(x.double(), dy.double(), w.double(), eps32)
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(gw, *want["weight"], F32, "grad_weight")
    if b is None:
        assert gb is None
    else:
        R.check(gb, *want["bias"], F32, "grad_bias")
    return out, mean, rstd, grad, gw, gb


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,d", NORM_SHAPES)
def test_layer_norm(ga, t, d, dtype):
    for wtype, bias in ((dtype, True), (F32, False)):
        _check_norm(ga, *_norm_case(t, d, dtype, wtype, t + d, bias), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(3, 0), (8, 0), (0, 1), (24, 8)])
@pytest.mark.parametrize("d", [40, 1024])
def test_layer_norm_layouts(ga, d, pad, shift, dtype):
    x, w, b, dy = _norm_case(37, d, dtype, dtype, 11)
    _check_norm(ga, x, w, b, dy, dtype, xd=_strided(x, pad, shift), dyd=_strided(dy, pad, shift))


def test_layer_norm_parameters_off_alignment(ga):
    x, w, b, dy = _norm_case(19, 512, BF16, BF16, 12)
    wd, bd = (torch.cat([v[:1], v]).cuda()[1:] for v in (w, b))
    out, mean, rstd = ga.layer_norm(x.cuda(), wd, bd)
    ref, rmean, rrstd = ga.layer_norm(x.cuda(), w.cuda(), b.cuda())
    want = R.layer_norm(x.double(), w.double(), b.double(), float(torch.tensor(1e-5)))
    R.check(out, *want["out"], BF16, "out")
    grad = ga.layer_norm_backward(dy.cuda(), x.cuda(), wd, mean, rstd)
    for a, c, key, t in zip(grad, ga.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rmean, rrstd),
                            ("grad", "weight", "bias"), (BF16, F32, F32)):
        want = R.layer_norm_backward(x.double(), dy.double(), w.double(), float(torch.tensor(1e-5)))
        R.check(a, *want[key], t, key)
        R.check(c, *want[key], t, key)


@pytest.mark.parametrize("d", [1, 8, 96, 33])
def test_layer_norm_constant_rows(ga, d):
    # variance 0: the row is the bias, and its gradient is finite
    x = torch.full((4, d), 3.0, dtype=BF16, device="cuda")
    w = torch.ones(d, dtype=BF16, device="cuda")
    b = torch.full((d,), 0.5, dtype=BF16, device="cuda")
    out, mean, rstd = ga.layer_norm(x, w, b)
    assert (out == 0.5).all() and (mean == 3).all()
    grad, gw, gb = ga.layer_norm_backward(torch.ones_like(x), x, w, mean, rstd)
    assert (grad == 0).all() and (gw == 0).all() and (gb == 4).all()


def test_layer_norm_no_rows(ga):
    x = torch.empty(0, 24, dtype=F32, device="cuda")
    w = torch.ones(24, device="cuda")
    out, mean, rstd = ga.layer_norm(x, w)
    assert out.shape == (0, 24) and mean.shape == rstd.shape == (0,)
    grad, gw, gb = ga.layer_norm_backward(x, x, w, mean, rstd)
    assert grad.shape == (0, 24) and (gw == 0).all() and (gb == 0).all()


def test_layer_norm_nan_stays_in_its_row(ga):
    x, w, b, dy = _norm_case(9, 256, BF16, BF16, 13)
    x[4, 7] = float("nan")
    xd = x.cuda()
    out, mean, rstd = ga.layer_norm(xd, w.cuda(), b.cuda())
    grad, gw, gb = ga.layer_norm_backward(dy.cuda(), xd, w.cuda(), mean, rstd)
    for t in (out, grad):
        assert torch.isnan(t).any(1).tolist() == [i == 4 for i in range(9)]
    assert torch.isnan(gw).all() and not torch.isnan(gb).any()


# -------------------------------------------------------------- balance loss

def _check_balance(ga, logits, ids, live, coef=0.25, view=None):
    """`logits`, `ids`, `live` on the CPU; `view`: the device logits to pass instead."""
    dtype = logits.dtype
    want = R.balance(logits.double(), ids.long(), live, coef)
    dev = logits.cuda() if view is None else view
    lv = live.cuda() if live is not None else None
    kept = ga.moe_balance_loss(dev, ids.cuda(), coef, live=lv)
    assert torch.equal(kept.counts.cpu(), want["counts"]) and kept.tokens.item() == want["tokens"]
    # probabilities: the exponent of a logit far below the maximum is rounded at its size
    R.check(kept.mean_p, want["mean_p"][0], 4 * want["mean_p"][1], F32, "mean_p")
    R.check(kept.loss, want["loss"][0], 4 * want["loss"][1], F32, "loss")
    up = torch.tensor([1.5], device="cuda")
    grad = ga.moe_balance_loss_backward(up, dev, kept, live=lv)
    R.check(grad, 1.5 * want["grad"][0], 6 * want["grad"][1], dtype, "grad")
    return kept, grad


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (3, 5, 1), (64, 128, 8), (1000, 60, 4),
                                   (257, 160, 6), (333, 33, 3), (2000, 512, 8), (50, 1000, 2),
                                   (77, 1024, 40), (5000, 16, 2), (300, 256, 8)])
def test_balance(ga, t, e, k, dtype):
    logits = (1.5 * _randn(t, e, seed=t) + 0.5 * _randn(1, e, seed=e)).to(dtype)
    ids = torch.randint(0, e, (t, k), generator=torch.Generator().manual_seed(t + k))
    live = _randn(t, seed=3) > -0.5
    _check_balance(ga, logits, ids, None)
    _check_balance(ga, logits, ids.int(), live)
    _check_balance(ga, logits, ids, live.to(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(3, 0), (8, 0), (0, 1), (24, 8)])
def test_balance_layouts(ga, pad, shift, dtype):
    logits = _randn(70, 64, seed=4).to(dtype)
    ids = torch.randint(0, 64, (70, 2), generator=torch.Generator().manual_seed(5))
    _check_balance(ga, logits, ids, None, view=_strided(logits, pad, shift))


@pytest.mark.parametrize("e", [8, 48, 128])
def test_balance_masked_experts_and_tokens(ga, e):
    logits = _randn(40, e, seed=6)
    logits[:, 1] = -float("inf")                 # an expert that is out
    logits[3, :] = -float("inf")                 # a token with none left
    logits[4] *= 20
    ids = torch.randint(-2, e + 3, (40, 2), generator=torch.Generator().manual_seed(7))
    live = torch.ones(40, dtype=torch.bool)
    kept, grad = _check_balance(ga, logits, ids, live)
    assert (grad[3] == 0).all() and (grad[:, 1] == 0).all()
    live[5], live[6] = False, False
    logits[5, 2], logits[6, :] = float("nan"), float("inf")      # padding may hold anything
    ids[5, 0], ids[6, 0] = 1 << 40, -(1 << 40)
    kept, grad = _check_balance(ga, logits.nan_to_num(7.0, posinf=7.0, neginf=-float("inf")), ids,
                                live, view=logits.cuda())
    assert (grad[5:7] == 0).all()
    kept, grad = _check_balance(ga, logits.nan_to_num(7.0, 7.0, -7.0), ids,
                                torch.zeros(40, dtype=torch.bool), view=logits.cuda())
    assert kept.loss.item() == 0 and (kept.counts == 0).all() and (grad == 0).all()


def test_balance_no_tokens_and_nan(ga):
    ids = torch.zeros(0, 2, dtype=torch.int64)
    kept = ga.moe_balance_loss(torch.zeros(0, 24, device="cuda"), ids.cuda(), 1.0)
    assert kept.loss.item() == 0 and kept.tokens.item() == 0 and (kept.counts == 0).all()
    assert ga.moe_balance_loss_backward(torch.ones(1, device="cuda"),
                                        torch.zeros(0, 24, device="cuda"), kept).shape == (0, 24)
    logits = _randn(5, 24, seed=8).cuda()
    logits[2, 3] = float("nan")
    kept = ga.moe_balance_loss(logits, torch.zeros(5, 1, dtype=torch.int64).cuda(), 1.0)
    grad = ga.moe_balance_loss_backward(torch.ones(1, device="cuda"), logits, kept)
    assert torch.isnan(kept.loss).all()
    assert torch.isnan(grad).all(1).tolist() == [i == 2 for i in range(5)]


# ------------------------------------------------- streams, graphs, far offsets

def _everything(ga, x, z, nx, w, logits, ids, stream=None):
    """Every operator once; a flat list of the outputs."""
    got = []
    dy = x[:, :x.shape[1] // 2]
    for name in ("silu", "gelu"):
        forward, backward = _ops(ga, name)
        out, kept = forward(x, stream=stream)
        flat = dy.contiguous() if stream is None and dy.is_cuda else dy
        got += [out, *kept[:2], *backward(flat, kept, recompute=True, stream=stream)]
    out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z, stream=stream)
    got += [out, *kept, *ga.gelu_and_mul_sparse_backward(dy, kept, z, recompute=True, stream=stream),
            ga.checkpoint_values(kept, stream=stream)]
    norm = ga.layer_norm(nx, w, w, stream=stream)
    got += [*norm, *ga.layer_norm_backward(nx, nx, w, norm[1], norm[2], stream=stream)]
    kept = ga.moe_balance_loss(logits, ids, 0.5, stream=stream)
    one = torch.ones(1, dtype=F32, device="cuda")
    return got + [*kept[:4], ga.moe_balance_loss_backward(one, logits, kept, stream=stream)]


def _inputs(seed=0):
    return (_gated(200, 768, BF16, seed), 1.0, _randn(900, 2048, seed=seed + 1).to(BF16).cuda(),
            _randn(2048, seed=seed + 2).cuda(), _randn(3000, 64, seed=seed + 3).cuda(),
            torch.randint(0, 64, (3000, 4), generator=torch.Generator().manual_seed(seed)).cuda())


def test_same_bits_again_and_on_another_stream(ga):
    args = _inputs()
    first = _everything(ga, *args)
    for a, b in zip(first, _everything(ga, *args)):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):          # what a call allocates must not be handed out again too early
        other = _everything(ga, *args, stream=s)
        torch.full((1 << 22,), 3.0, device="cuda")
    s.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)


def test_graph_capture(ga):
    args = _inputs(3)
    want = _everything(ga, *args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _everything(ga, *args)
    for t in got:
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_host_rows_in_place(ga):
    x = _gated(20, 96, BF16, 5)
    xh = x.cpu().pin_memory()
    out, kept = ga.silu_and_mul_checkpoint(xh)
    want, wkept = ga.silu_and_mul_checkpoint(x)
    torch.cuda.synchronize()
    assert not out.is_cuda and torch.equal(out, want.cpu())
    assert torch.equal(kept.codes, wkept.codes.cpu())


def test_everything_on_host_rows(ga):
    # page-locked rows are read and written in place, to the same bits
    args = _inputs(7)
    want = _everything(ga, *args)
    host = [a.cpu().pin_memory() if isinstance(a, torch.Tensor) else a for a in args]
    got = _everything(ga, *host)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert not b.is_cuda and torch.equal(a.cpu(), b)


def test_more_than_2_to_31_vectors(ga):
    # rows of one vector, more of them than 32-bit indexes hold
    m, d = (1 << 30) // 2 + 5, 8
    x = torch.zeros((m, 2 * d), dtype=BF16, device="cuda")
    x[-3:] = _gated(3, d, BF16, 8)
    tail = x[-3:].clone()
    out, kept = ga.silu_and_mul_checkpoint(x)
    want, wkept = ga.silu_and_mul_checkpoint(tail)
    assert torch.equal(out[-3:], want) and (out[:-3:1 << 20] == 0).all()
    assert torch.equal(kept.codes[-3:], wkept.codes) and torch.equal(kept.scales[-3:], wkept.scales)
    del x
    assert torch.equal(ga.silu_and_mul_backward(out, kept)[-3:],
                       ga.silu_and_mul_backward(out[-3:].clone(), wkept))
    assert torch.equal(ga.checkpoint_values(kept)[-3:], ga.checkpoint_values(wkept))


@pytest.mark.parametrize("d", [16384, 16385])
def test_offsets_past_32_bits(ga, d):
    # 2^31 elements and more in one tensor: the last rows are those of a short call
    m = (1 << 31) // (2 * d) + 40
    x = torch.zeros((m, 2 * d), dtype=BF16, device="cuda")
    x[-3:] = _gated(3, d, BF16, 6)
    dy = torch.zeros((m, d), dtype=BF16, device="cuda")
    dy[-3:] = _randn(3, d, seed=7).to(BF16).cuda()
    tail, dtail = x[-3:].clone(), dy[-3:].clone()
    out, kept = ga.silu_and_mul_checkpoint(x)
    want, wkept = ga.silu_and_mul_checkpoint(tail)
    assert torch.equal(out[-3:], want) and torch.equal(kept.codes[-3:], wkept.codes)
    assert torch.equal(ga.silu_and_mul_backward(dy, kept)[-3:], ga.silu_and_mul_backward(dtail, wkept))
    assert torch.equal(ga.checkpoint_values(kept)[-3:], ga.checkpoint_values(wkept))
    out, kept = ga.gelu_and_mul_sparse_checkpoint(x, 1.0)
    want, wkept = ga.gelu_and_mul_sparse_checkpoint(tail, 1.0)
    assert torch.equal(out[-3:], want) and torch.equal(kept.codes[-3:], wkept.codes)
    assert torch.equal(ga.gelu_and_mul_sparse_backward(dy, kept, 1.0)[-3:],
                       ga.gelu_and_mul_sparse_backward(dtail, wkept, 1.0))
    del out, kept, want, wkept
    w = torch.ones(2 * d, dtype=BF16, device="cuda")
    got, mean, rstd = ga.layer_norm(x, w)
    want, wmean, wrstd = ga.layer_norm(tail, w)
    # the rows may be split over the CTAs otherwise: values, not bits
    assert torch.allclose(got[-3:].float(), want.float(), rtol=2.0 ** -7, atol=1e-6)
    grad = ga.layer_norm_backward(x, x, w, mean, rstd, bias=False)[0]
    wgrad = ga.layer_norm_backward(tail, tail, w, wmean, wrstd, bias=False)[0]
    assert torch.allclose(grad[-3:].float(), wgrad.float(), rtol=2.0 ** -6, atol=1e-4)


def test_guard_bands(ga):
    # nothing outside the outputs is written, whatever their alignment
    lib, s = ga.load_library(), torch.cuda.current_stream().cuda_stream
    for m, d in ((3, 37), (5, 64), (2, 4099), (4, 2048)):
        nb = -(-d // 32)
        x = _gated(m, d, BF16, 9)
        dy = _randn(m, d, seed=1).to(BF16).cuda()
        sizes = {"out": 2 * m * d, "codes": 2 * m * d, "scales": 2 * m * nb, "grad": 4 * m * d,
                 "again": 2 * m * d}
        for off in (0, 2, 16):
            bufs = {k: torch.full((n + 128,), 0xA5, dtype=torch.uint8, device="cuda")
                    for k, n in sizes.items()}
            p = {k: ctypes.c_void_p(b.data_ptr() + 64 + off) for k, b in bufs.items()}
            assert lib.gelu_and_mul_checkpoint(p["out"], p["codes"], p["scales"], x.data_ptr(), m,
                                               d, 2 * d, ga.BF16, None, s) == 0
            assert lib.gelu_and_mul_backward(p["grad"], p["again"], dy.data_ptr(), p["codes"],
                                             p["scales"], m, d, d, ga.BF16, None, s) == 0
            for k, b in bufs.items():
                head, tail = b[:64 + off], b[64 + off + sizes[k]:]
                assert (head == 0xA5).all() and (tail == 0xA5).all(), (k, m, d, off)
            out, kept = ga.gelu_and_mul_checkpoint(x)
            mine = bufs["out"][64 + off:64 + off + sizes["out"]].cpu().view(BF16).view(m, d)
            assert torch.equal(mine, out.cpu())
