"""The training operators at the ends of their ranges: what their formulas give where the
arithmetic could lose it, and every kernel that the sizes choose, against the 64-bit forms of
tests/training_ref.py (which derives the bounds)."""
import pytest
import torch

import workloads as W
from tests import training_ref as R
from tests.gpu_util import require_gpu
from tests.test_training_gpu import (BF16, DTYPES, F16, F32, _check_balance, _check_norm,
                                     _check_sparse_forward, _gated, _norm_case, _ops, _randn)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ga():
    return require_gpu()


def _chosen(t, e, k, seed):
    return torch.randint(0, e, (t, k), generator=torch.Generator().manual_seed(seed))


# -------------------------------------------------------------- balance loss

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e", [(1, 1), (13, 8), (700, 60), (14383, 8), (3000, 128)])
def test_balance_equal_counts_have_no_gradient(ga, t, e, dtype):
    # every token chooses every expert: the loss is the coefficient, whatever the logits, and the
    # gradient exactly 0
    logits = (1.5 * _randn(t, e, seed=t)).to(dtype)
    ids = torch.stack([torch.randperm(e, generator=torch.Generator().manual_seed(i % 7))
                       for i in range(t)])
    kept, grad = _check_balance(ga, logits, ids, _randn(t, seed=2) > -0.5)
    assert (grad == 0).all()
    kept, grad = _check_balance(ga, logits, ids, None, coef=0.25)
    assert (grad == 0).all() and abs(kept.loss.item() - 0.25) < 1e-5


# rows: the one-launch cluster, and the two launches of a longer batch
LARGE = {F16: [-65504.0, 65504.0, -3e4], BF16: [torch.finfo(BF16).min, torch.finfo(BF16).max,
                                                -1e30, 1e30, -1e10, 1e10],
         F32: [torch.finfo(F32).min, torch.finfo(F32).max, -1e30, 1e30, -1e10, 1e10, 12345678.0]}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [7, 901])
@pytest.mark.parametrize("e", [1, 8, 24, 60, 128, 512, 1000])
def test_balance_large_logits(ga, t, e, dtype):
    # a row of one value, the type's lowest (a mask's) or another far from 0: every expert's
    # probability is 1 / E
    value = torch.tensor([LARGE[dtype][i % len(LARGE[dtype])] for i in range(t)])
    logits = value[:, None].expand(t, e).to(dtype).contiguous()
    kept, _ = _check_balance(ga, logits, _chosen(t, e, 2, t), None)
    assert torch.allclose(kept.mean_p.cpu(), torch.full((e,), 1 / e), rtol=1e-5)
    # some experts at the lowest value beside ordinary ones: those have probability 0
    logits = _randn(t, e, seed=e).to(dtype)
    logits[:, 1::3] = torch.finfo(dtype).min
    _, grad = _check_balance(ga, logits, _chosen(t, e, 2, t), None)
    assert (grad[:, 1::3] == 0).all()


@pytest.mark.parametrize("t", [7, 901])
@pytest.mark.parametrize("e", [8, 60, 128])
def test_balance_logits_around_a_large_value(ga, t, e):
    # differences that fp32 holds exactly, far from 0
    steps = torch.randint(-12, 1, (t, e), generator=torch.Generator().manual_seed(e)).float()
    for base in (-2.0 ** 23, 2.0 ** 23, 2.0 ** 22 + 0.5):
        _check_balance(ga, steps + base, _chosen(t, e, 2, t), None)


@pytest.mark.parametrize("up", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("t,e", [(40, 8), (40, 60), (901, 128), (901, 33)])
def test_balance_rows_that_are_not_live_with_a_loss_gradient_that_is_not_finite(ga, t, e, up):
    # the gradient of a loss scale that overflowed: 0 in rows that are not live all the same
    logits = _randn(t, e, seed=t).cuda()
    live = torch.arange(t, device="cuda") % 3 != 1
    kept = ga.moe_balance_loss(logits, _chosen(t, e, 1, t).cuda(), 0.5, live=live)
    for on in (live, torch.zeros_like(live)):
        grad = ga.moe_balance_loss_backward(torch.full((1,), up, device="cuda"), logits, kept, live=on)
        assert (grad[~on] == 0).all() and not torch.isfinite(grad[on]).any()


# ---------------------------------------------------------------- layer norm

# rows that clusters of two and four share: fewer and more of them than clusters on the GPU
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,d", [(1, 8200), (3, 16384), (200, 9000), (90, 16400), (1, 24576),
                                 (170, 32768)])
def test_layer_norm_rows_that_a_cluster_shares(ga, t, d, dtype):
    for wtype, bias in ((dtype, True), (F32, False)):
        _check_norm(ga, *_norm_case(t, d, dtype, wtype, t + d, bias), dtype)


def test_layer_norm_rows_that_a_cluster_shares_again(ga):
    # the same bits every time, one call behind the other
    x, w, _, dy = _norm_case(300, 20480, BF16, F32, 5)
    x, w, dy = x.cuda(), w.cuda(), dy.cuda()
    _, mean, rstd = ga.layer_norm(x, w)
    first = ga.layer_norm_backward(dy, x, w, mean, rstd)
    for got in [ga.layer_norm_backward(dy, x, w, mean, rstd) for _ in range(20)]:
        for a, b in zip(first, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1e-20, 1e-15, 1e15, 1e20])
@pytest.mark.parametrize("t,d", [(5, 64), (40, 2048), (3, 8192), (5, 301), (9, 2047), (2, 16384),
                                 (2, 20000), (2, 40001)])
def test_layer_norm_backward_of_small_and_large_deviations(ga, t, d, scale, dtype):
    # 1 / std whose square fp32 does not hold; gradients that follow the row, so that the mean of
    # g hat is about 1
    x = (scale * _randn(t, d, seed=d)).to(dtype)
    dy = (x.float() / scale + 0.5 * _randn(t, d, seed=d + 1)).to(dtype)
    w = 1 + 0.2 * _randn(d, seed=d + 2)
    want = R.layer_norm(x.double(), w.double(), None, 0.0)
    mean, rstd = (want[k][0].to(F32).cuda() for k in ("mean", "rstd"))
    grad, gw, gb = ga.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    want = R.layer_norm_backward(x.double(), dy.double(), w.double(), 0.0)
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(gw, *want["weight"], F32, "grad_weight")
    R.check(gb, *want["bias"], F32, "grad_bias")


# --------------------------------------------------------------- checkpoints

# one per lane and in vectors, of every kernel: rows in registers, in the ring, read again
@pytest.mark.parametrize("dtype,m,d", [(F32, 3, 257), (F32, 3, 1000), (F32, 2, 1001), (F32, 2, 2048),
                                       (F32, 2, 4096), (F32, 2, 8193), (F32, 2, 16384),
                                       (F32, 2, 20001), (F32, 2, 40000), (F16, 2, 32760), (F16, 3, 12001),
                                       (F16, 2, 32761), (F16, 2, 40000), (BF16, 2, 70000),
                                       (F16, 2437, 1032), (F16, 613, 4104), (F16, 311, 16376)])
def test_sparse_constant_rows(ga, m, d, dtype):
    # constants of many digits, whose sums are rounded: the deviation is 0 all the same, nothing
    # passes, and the gradients are 0
    value = torch.tensor([2.5841505, 2.71828, -0.1, 1 / 3, 77.7, 1e-3, 12345.678])
    gate = value[torch.arange(m) % len(value)][:, None].expand(m, d)
    x = torch.cat([gate, _randn(m, d, seed=d)], 1).to(dtype).cuda()
    dy = torch.ones(m, d, dtype=dtype, device="cuda")
    for z in (0.0, W.Z95, -1.0):
        out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z)
        assert (kept.std == 0).all() and (kept.codes[:, :d] == 0).all() and (out == 0).all()
        assert (ga.gelu_and_mul_sparse_backward(dy, kept, z) == 0).all()


@pytest.mark.parametrize("dtype,m,d", [(F32, 7, 257), (F32, 6, 1000), (F32, 6, 16384),
                                       (F16, 2437, 1032), (F16, 2, 40000)])
def test_sparse_rows_constant_but_for_one_element(ga, m, d, dtype):
    # the one element may be the first, the last or any other
    x = _gated(m, d, dtype, 7)
    x[:, :d] = 0.7
    at = torch.tensor([0, d - 1, d // 2, 1, 8, 33])[torch.arange(m) % 6].cuda()
    x[torch.arange(m, device="cuda"), at] = 0.9
    for z in (0.0, 1.0):
        out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z)
        _check_sparse_forward(x.double().cpu(), d, z, dtype, out, kept)
        assert (kept.std > 0).all()
        assert (kept.codes[:, :d] > 0).sum(1).eq(1).all()


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 37])
def test_small_up_values_beside_large_gates(ga, d, dtype, name):
    # an up half at the lower end of the normal range, whose products with the gate are normal:
    # no factor on the way may take them below it
    gates = torch.tensor([0.5, 3.0, 8.0, 13.0, 22.5, 30.0, 60.0, 500.0, -0.5, -3.0, -20.0, -70.0])
    gate = gates[:, None].expand(len(gates), d)
    up = 1.2e-38 * (1 + _randn(len(gates), d, seed=1).abs())
    x = torch.cat([gate, up], 1).to(dtype)
    forward, backward = _ops(ga, name)
    out, kept = forward(x.cuda())
    xr = x.double()
    a, _, _, grow = R.act(name, xr[:, :d])
    R.check(out, a * xr[:, d:], (a * xr[:, d:]).abs() * grow, dtype, "out")
    dy = _randn(len(gates), d, seed=2).to(dtype)
    want = R.act_backward(name, R.values(kept.codes, kept.scales), dy.double())
    grad, again = backward(dy.cuda(), kept, recompute=True)
    R.check(grad, *want["grad"], dtype, "grad")
    R.check(again, *want["out"], dtype, "recomputed out")


@pytest.mark.parametrize("d", [0, -1, 9, 1 << 40, 1 << 62, (1 << 63) - 1])
def test_widths_that_the_rows_do_not_hold(ga, d):
    x = torch.zeros(0, 16, dtype=BF16, device="cuda")
    for call in (lambda: ga.silu_and_mul_checkpoint(x, d=d),
                 lambda: ga.gelu_and_mul_sparse_checkpoint(x, 1.0, d=d)):
        with pytest.raises(ValueError):
            call()
