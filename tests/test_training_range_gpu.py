"""The training operators at the ends of their ranges: what their formulas give where the
arithmetic could lose it, and every kernel that the sizes choose, against the 64-bit forms of
tests/training_ref.py (which derives the bounds)."""
import ctypes

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


@pytest.mark.parametrize("e", [8, 24, 60])
def test_balance_gradient_of_counts_past_2_to_24(ga, e):
    # counts that fp32 does not hold, a few choices apart
    t, k, up = 5, 4, 2.0 ** 40
    logits = _randn(t, e, seed=e)
    counts = (1 << 31) // e - 64 + torch.randint(-3, 4, (e,), generator=torch.Generator().manual_seed(e))
    n = int(counts.sum()) // k
    kept = ga.BalanceLoss(torch.zeros(1).cuda(), counts.int().cuda(),
                          torch.tensor([n], dtype=torch.int32).cuda(), torch.zeros(e).cuda(), k, 1.0)
    grad = ga.moe_balance_loss_backward(torch.full((1,), up).cuda(), logits.cuda(), kept)
    p = torch.softmax(logits.double(), 1)
    c = counts.double() - counts.double().mean()
    scale = up * e / (n * n * k)
    mag = scale * p * (c.abs() + 1 + (p * (c.abs() + 1)).sum(1, keepdim=True))
    R.check(grad, scale * p * (c - (p * c).sum(1, keepdim=True)), 6 * mag, F32, "grad")


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


@pytest.mark.parametrize("dtype,t,d", [(F32, 7, 64), (F32, 7, 200), (F32, 7, 1000), (F32, 7, 2048),
                                       (F32, 7, 2047), (F32, 7, 4097), (F32, 7, 16384), (F32, 7, 20000),
                                       (F32, 7, 40001), (F16, 7, 1001), (F16, 9, 12345), (F16, 7, 16383),
                                       (F16, 7, 40000), (BF16, 7, 16383), (BF16, 7, 70000)])
def test_layer_norm_rows_of_one_value(ga, t, d, dtype):
    # values of many digits, whose sums are rounded: the mean is the value, the deviation 0 and
    # the output the bias, with eps far below the value's rounding too
    value = torch.tensor([2.5841505, 2.71828, -0.1, 1 / 3, 77.7, 1e-3, 12345.678])
    x = value[torch.arange(t) % 7][:, None].expand(t, d).to(dtype).cuda()
    w, b = 1 + _randn(d, seed=1).cuda(), _randn(d, seed=2).cuda()
    out, mean, rstd = ga.layer_norm(x.contiguous(), w, b, eps=1e-5)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(out, b.to(dtype).expand(t, d))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("dtype,t,d", [(F32, 6, 64), (F32, 6, 2047), (F32, 6, 16384), (F32, 6, 20000),
                                       (F16, 6, 16383), (F32, 6, 40001)])
def test_layer_norm_rows_of_one_value_but_for_one_element(ga, t, d, dtype):
    x = torch.full((t, d), 0.7)
    x[torch.arange(t), torch.tensor([0, d - 1, d // 2, 1, 8, 33])] = 0.9
    _check_norm(ga, x.to(dtype), *_norm_case(t, d, dtype, F32, 3)[1:], dtype)


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


# ----------------------------------- the kernels of every class of widths and batches

# widths in whole vectors between those of the other tests: a few rows, more than the shares
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,d", [(3, 2056), (3, 4096), (700, 4096), (320, 3000), (2, 6144), (170, 4104),
                                 (2, 8208), (170, 12288), (160, 16384)])
def test_layer_norm_widths(ga, t, d, dtype):
    for wtype, bias in ((dtype, True), (F32, False)):
        _check_norm(ga, *_norm_case(t, d, dtype, wtype, t + d, bias), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,d", [(33, 4095), (170, 10001), (160, 16383)])
def test_layer_norm_widths_off_a_boundary(ga, t, d, dtype):
    _check_norm(ga, *_norm_case(t, d, dtype, F32, t + d, True), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", [(3, 1032), (5, 2048), (3, 2056), (700, 4096), (2, 4104), (3, 8200),
                                 (40, 12288), (160, 16384), (3, 24576)])
def test_sparse_widths(ga, m, d, dtype):
    for z in (0.0, W.Z95):
        x = _gated(m, d, dtype, d + m)
        out, kept = ga.gelu_and_mul_sparse_checkpoint(x, z)
        _check_sparse_forward(x.double().cpu(), d, z, dtype, out, kept)
        dy = _randn(m, d, seed=d + 1).to(dtype)
        want = R.sparse_backward(R.values(kept.codes, kept.scales), dy.double(),
                                 kept.std.double().cpu(), z)
        grad, again = ga.gelu_and_mul_sparse_backward(dy.cuda(), kept, z, recompute=True)
        R.check(grad, *want["grad"], dtype, "grad")
        R.check(again, *want["out"], dtype, "recomputed out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,k", [(769, 1, 1), (900, 8, 2), (1100, 24, 2), (1300, 32, 4), (1000, 64, 4),
                                   (1000, 128, 8), (20000, 128, 8), (1200, 160, 6), (800, 256, 8),
                                   (2000, 384, 6), (900, 1000, 2), (900, 1024, 8), (800, 5, 2),
                                   (900, 100, 4), (800, 250, 3), (850, 500, 2), (850, 1001, 2)])
def test_balance_long_batches(ga, t, e, k, dtype):
    logits = (1.5 * _randn(t, e, seed=t) + 0.5 * _randn(1, e, seed=e)).to(dtype)
    ids = _chosen(t, e, k, t + k)
    _check_balance(ga, logits, ids, None)
    _check_balance(ga, logits, ids.int(), _randn(t, seed=3) > -0.5)


# ------------------------------------------------------ what the outputs end at

class _Guarded:
    """Output buffers with bands around them that must stay as they are."""

    def __init__(self, off, **sizes):
        self.off, self.sizes = off, sizes
        self.buf = {k: torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
                    for k, n in sizes.items()}

    def __getitem__(self, k):
        return ctypes.c_void_p(self.buf[k].data_ptr() + 256 + self.off)

    def check(self, what):
        for k, b in self.buf.items():
            end = 256 + self.off + self.sizes[k]
            assert (b[:256 + self.off] == 0xA5).all() and (b[end:] == 0xA5).all(), (k, *what)


@pytest.mark.parametrize("dtype,m,d", [(BF16, 3, 37), (BF16, 2, 1000), (BF16, 2, 4099), (F32, 3, 1001),
                                       (F32, 3, 8192), (BF16, 2437, 1032), (BF16, 311, 16376),
                                       (F16, 2, 40001)])
def test_guard_bands_sparse(ga, m, d, dtype):
    lib, s = ga.load_library(), torch.cuda.current_stream().cuda_stream
    x, dy, nb = _gated(m, d, dtype, 9), _randn(m, d, seed=1).to(dtype).cuda(), -(-d // 32)
    size, code = x.element_size(), {BF16: ga.BF16, F16: ga.F16, F32: ga.F32}[dtype]
    for off in (0, size, 32):
        g = _Guarded(off, out=size * m * d, codes=2 * m * d, scales=2 * m * nb, grad=2 * size * m * d,
                     again=size * m * d)
        f = _Guarded(0, std=4 * m, values=8 * m * d)
        assert lib.gelu_and_mul_sparse_checkpoint(g["out"], g["codes"], g["scales"], f["std"],
                                                  x.data_ptr(), m, d, 2 * d, 1.0, code, s) == 0
        assert lib.gelu_and_mul_sparse_backward(g["grad"], g["again"], dy.data_ptr(), g["codes"],
                                                g["scales"], f["std"], m, d, d, 1.0, code, s) == 0
        assert lib.gated_act_checkpoint_values(f["values"], g["codes"], g["scales"], m, d, ga.F32,
                                               s) == 0
        g.check((m, d, off))
        f.check((m, d, off))


@pytest.mark.parametrize("dtype,t,d", [(BF16, 3, 37), (BF16, 5, 301), (BF16, 700, 2047), (F32, 9, 1001),
                                       (F32, 3, 4096), (BF16, 3, 12345), (BF16, 2, 20000),
                                       (F16, 2, 40001)])
def test_guard_bands_layer_norm(ga, t, d, dtype):
    lib, s = ga.load_library(), torch.cuda.current_stream().cuda_stream
    x, w, b, dy = (v.cuda() for v in _norm_case(t, d, dtype, F32, 3))
    size, code = x.element_size(), {BF16: ga.BF16, F16: ga.F16, F32: ga.F32}[dtype]
    need = lib.layer_norm_backward_workspace_bytes(t, d)
    for off in (0, size, 16):
        g = _Guarded(off, out=size * t * d, grad=size * t * d)
        f = _Guarded(0, mean=4 * t, rstd=4 * t, gw=4 * d, gb=4 * d, ws=need)
        assert lib.layer_norm(g["out"], f["mean"], f["rstd"], x.data_ptr(), w.data_ptr(), b.data_ptr(),
                              t, d, d, 1e-5, code, ga.F32, s) == 0
        assert lib.layer_norm_backward(g["grad"], f["gw"], f["gb"], dy.data_ptr(), x.data_ptr(),
                                       w.data_ptr(), f["mean"], f["rstd"], t, d, d, d, code, ga.F32,
                                       f["ws"], need, s) == 0
        g.check((t, d, off))
        f.check((t, d, off))


@pytest.mark.parametrize("dtype,t,e", [(BF16, 3, 8), (BF16, 40, 60), (F32, 901, 33), (F32, 900, 128),
                                       (F16, 900, 1000), (BF16, 5000, 5)])
def test_guard_bands_balance(ga, t, e, dtype):
    lib, s = ga.load_library(), torch.cuda.current_stream().cuda_stream
    x, ids = _randn(t, e, seed=1).to(dtype).cuda(), _chosen(t, e, 2, 1).cuda()
    size, code = x.element_size(), {BF16: ga.BF16, F16: ga.F16, F32: ga.F32}[dtype]
    need = lib.moe_balance_loss_workspace_bytes(t, e)
    one = torch.ones(1, device="cuda")
    for off in (0, size, 32):
        g = _Guarded(off, grad=size * t * e)
        f = _Guarded(0, loss=4, counts=4 * e, tokens=4, p=4 * e, ws=need)
        assert lib.moe_balance_loss(f["loss"], f["counts"], f["tokens"], f["p"], x.data_ptr(),
                                    ids.data_ptr(), None, t, e, 2, e, code, 1, 0.5, f["ws"], need,
                                    s) == 0
        assert lib.moe_balance_loss_backward(g["grad"], one.data_ptr(), x.data_ptr(), f["counts"],
                                             f["tokens"], None, t, e, 2, e, code, 0.5, s) == 0
        g.check((t, e, off))
        f.check((t, e, off))


# -------------------------------------------- indexes past 32 bits, kernel by kernel

def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB of device memory")


def _tail_kept(ga, d):
    x = _gated(3, d, BF16, 8)
    return x, *ga.silu_and_mul_checkpoint(x)


def test_more_than_2_to_31_vectors_of_values(ga):
    # 2 d / 8 vectors per row: 2^31 and more in 2^30 rows of d = 8
    _room(80)
    m, d = (1 << 30) + 5, 8
    _, _, tail = _tail_kept(ga, d)
    codes = torch.zeros((m, 2 * d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((m, 2), dtype=torch.uint8, device="cuda")
    codes[-3:], scales[-3:] = tail.codes, tail.scales
    got = ga.checkpoint_values(ga.Checkpoint(codes, scales))
    assert torch.equal(got[-3:], ga.checkpoint_values(tail)) and (got[:-3:1 << 20] == 0).all()


def test_more_than_2_to_31_vectors_of_gradients(ga):
    # d / 8 vectors per row: 2^31 rows and more of d = 8
    _room(180)
    m, d = (1 << 31) + 5, 8
    _, _, tail = _tail_kept(ga, d)
    codes = torch.zeros((m, 2 * d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((m, 2), dtype=torch.uint8, device="cuda")
    codes[-3:], scales[-3:] = tail.codes, tail.scales
    dy = torch.zeros((m, d), dtype=BF16, device="cuda")
    dy[-3:] = _randn(3, d, seed=7).to(BF16).cuda()
    short = ga.silu_and_mul_backward(dy[-3:].clone(), tail)
    got = ga.silu_and_mul_backward(dy, ga.Checkpoint(codes, scales))
    assert torch.equal(got[-3:], short) and (got[:-3:1 << 20] == 0).all()
    del got, dy, codes, scales
    torch.cuda.empty_cache()


def test_more_than_2_to_31_blocks_element_by_element(ga):
    # one block per row: 2^31 rows and more of d = 1
    _room(60)
    m, d = (1 << 31) + 5, 1
    tail, want, wkept = _tail_kept(ga, d)
    x = torch.zeros((m, 2 * d), dtype=BF16, device="cuda")
    x[-3:] = tail
    out, kept = ga.silu_and_mul_checkpoint(x)
    del x
    assert torch.equal(out[-3:], want) and (out[:-3:1 << 20] == 0).all()
    assert torch.equal(kept.codes[-3:], wkept.codes) and torch.equal(kept.scales[-3:], wkept.scales)
    short, again = ga.silu_and_mul_backward(want, wkept, recompute=True)
    got, gagain = ga.silu_and_mul_backward(out, kept, recompute=True)
    assert torch.equal(got[-3:], short) and torch.equal(gagain[-3:], again)
    del got, gagain, out
    assert torch.equal(ga.checkpoint_values(kept)[-3:], ga.checkpoint_values(wkept))
