"""Refusals of the training operators: sizes, strides, types, pointers, workspaces.  No call
here launches a kernel: each fails its checks before any CUDA call, or is a zero-row no-op."""
import pytest
import torch

import gated_activation_gb300 as ga
from gated_activation_gb300 import build as gbuild

A, B, C, D, E, F = (0x100000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    if not gbuild.up_to_date():
        gbuild.build()
    return ga.load_library()


def test_scale_bytes(lib):
    got = [lib.gated_act_checkpoint_scales(d) for d in (-1, 0, 1, 32, 33, 768, 1 << 30)]
    assert got == [0, 0, 2, 2, 4, 48, 1 << 26]


def _forward(lib, name, out=A, codes=B, scales=C, inp=D, m=4, d=8, rs=16, dtype=ga.BF16, n=None):
    if name == "sparse":
        return lib.gelu_and_mul_sparse_checkpoint(out, codes, scales, E, inp, m, d, rs, 1.0, dtype,
                                                  None)
    return getattr(lib, name + "_and_mul_checkpoint")(out, codes, scales, inp, m, d, rs, dtype, n,
                                                      None)


def _backward(lib, name, grad_in=A, out=None, grad=B, codes=C, scales=D, m=4, d=8, gs=8,
              dtype=ga.BF16, n=None, std=E):
    if name == "sparse":
        return lib.gelu_and_mul_sparse_backward(grad_in, out, grad, codes, scales, std, m, d, gs,
                                                1.0, dtype, None)
    return getattr(lib, name + "_and_mul_backward")(grad_in, out, grad, codes, scales, m, d, gs,
                                                    dtype, n, None)


@pytest.mark.parametrize("name", ["silu", "gelu", "sparse"])
def test_checkpoint_refusals(lib, name):
    f = lambda **k: _forward(lib, name, **k)  # noqa: E731
    assert f(m=-1) == f(d=0) == f(d=-8) == ga.ERR_SIZE
    assert f(rs=15) == f(rs=0) == ga.ERR_STRIDE
    assert f(dtype=3) == f(dtype=-1) == ga.ERR_DTYPE
    assert f(d=(1 << 30) + 1, rs=1 << 32) == f(m=1 << 41) == f(m=1 << 40, rs=1 << 40) \
        == ga.ERR_TOO_LARGE
    assert f(m=0, out=None, inp=None) == ga.OK
    for missing in ("out", "codes", "scales", "inp"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(out=A + 1) == f(inp=D + 1) == f(out=A + 2, dtype=ga.F32) == ga.ERR_ALIGN
    # out spans 64 bytes, codes 64, scales 8, in 128
    assert f(out=D + 126) == f(codes=D + 127) == f(codes=A + 63) == f(scales=B + 63) \
        == ga.ERR_OVERLAP
    b = lambda **k: _backward(lib, name, **k)  # noqa: E731
    assert b(m=-1) == b(d=0) == ga.ERR_SIZE and b(gs=7) == ga.ERR_STRIDE
    assert b(dtype=7) == ga.ERR_DTYPE and b(m=1 << 40, gs=1 << 40) == ga.ERR_TOO_LARGE
    assert b(m=0, grad_in=None, grad=None) == ga.OK
    for missing in ("grad_in", "grad", "codes", "scales"):
        assert b(**{missing: None}) == ga.ERR_NULL
    assert b(grad_in=A + 1) == b(out=F + 1) == b(grad=B + 1) == ga.ERR_ALIGN
    assert b(grad_in=B - 126) == b(out=A + 64) == b(out=B) == b(grad_in=C) == ga.ERR_OVERLAP
    if name == "sparse":
        assert b(std=None) == ga.ERR_NULL and b(std=E + 2) == ga.ERR_ALIGN
        assert b(grad_in=E) == ga.ERR_OVERLAP
    else:
        assert f(n=0x5002) == b(n=0x5002) == ga.ERR_ALIGN


def test_values_refusals(lib):
    v = lib.gated_act_checkpoint_values
    assert v(A, B, C, 4, 8, ga.F16, None) == v(A, B, C, 4, 8, 9, None) == ga.ERR_DTYPE
    assert v(A, B, C, -4, 8, ga.F32, None) == ga.ERR_SIZE
    assert v(A, None, C, 4, 8, ga.F32, None) == ga.ERR_NULL
    assert v(B, B, C, 4, 8, ga.F32, None) == ga.ERR_OVERLAP
    assert v(None, None, None, 0, 8, ga.F32, None) == ga.OK


def test_layer_norm_refusals(lib):
    def f(out=A, mean=B, rstd=C, x=D, w=E, b=F, t=4, d=8, rs=8, eps=1e-5, dt=ga.BF16, wt=ga.BF16):
        return lib.layer_norm(out, mean, rstd, x, w, b, t, d, rs, eps, dt, wt, None)

    assert f(t=-1) == f(d=0) == f(eps=-1e-9) == f(eps=float("nan")) == ga.ERR_SIZE
    assert f(rs=7) == ga.ERR_STRIDE
    assert f(dt=5) == f(wt=ga.F16) == f(dt=ga.F32, wt=ga.BF16) == ga.ERR_DTYPE
    assert f(d=1 << 31, rs=1 << 31) == f(t=1 << 40, rs=1 << 30) == ga.ERR_TOO_LARGE
    assert f(t=0, out=None, x=None, w=None) == ga.OK
    for missing in ("out", "mean", "rstd", "x", "w"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(mean=B + 2) == f(w=E + 1) == f(w=E + 2, wt=ga.F32) == ga.ERR_ALIGN
    assert f(out=D) == f(mean=C) == f(out=E - 62) == f(rstd=F) == ga.ERR_OVERLAP


def test_layer_norm_backward_refusals(lib):
    def f(gi=A, gw=B, gb=None, dy=C, x=D, w=E, mean=F, rstd=F + 64, t=4, d=8, rs=8, gs=8,
          dt=ga.BF16, wt=ga.F32, ws=0x900000, n=1 << 20):
        return lib.layer_norm_backward(gi, gw, gb, dy, x, w, mean, rstd, t, d, rs, gs, dt, wt, ws,
                                       n, None)

    need = lib.layer_norm_backward_workspace_bytes(4, 8)
    assert need >= 16 and lib.layer_norm_backward_workspace_bytes(0, 8) == 16
    assert f(t=-1) == f(d=0) == ga.ERR_SIZE
    assert f(rs=7) == f(gs=7) == ga.ERR_STRIDE
    assert f(wt=ga.F16) == ga.ERR_DTYPE
    assert f(n=need - 1) == ga.ERR_SCRATCH
    for missing in ("gi", "gw", "dy", "x", "w", "mean", "rstd", "ws"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(ws=0x900008) == f(gw=B + 2) == f(x=D + 1) == ga.ERR_ALIGN
    assert f(gi=C) == f(gw=E) == f(gb=B + 4) == f(ws=D) == f(gi=F) == ga.ERR_OVERLAP


def test_balance_refusals(lib):
    def f(loss=A, counts=A + 64, tokens=A + 256, p=A + 512, x=B, ids=C, live=None, t=4, e=8, k=2,
          ls=8, dt=ga.F32, wide=1, ws=D, n=1 << 20):
        return lib.moe_balance_loss(loss, counts, tokens, p, x, ids, live, t, e, k, ls, dt, wide,
                                    0.1, ws, n, None)

    need = lib.moe_balance_loss_workspace_bytes(4, 8)
    assert need >= 16 and need % 16 == 0
    assert f(t=-1) == f(e=0) == f(k=0) == ga.ERR_SIZE
    assert f(ls=7) == ga.ERR_STRIDE and f(dt=4) == ga.ERR_DTYPE
    assert f(e=1025, ls=2000) == f(t=1 << 30, k=4) == f(t=1 << 32) == ga.ERR_TOO_LARGE
    assert f(n=need - 1) == ga.ERR_SCRATCH
    for missing in ("loss", "counts", "tokens", "p", "x", "ids", "ws"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(ids=C + 4) == f(x=B + 2) == f(loss=A + 1) == ga.ERR_ALIGN
    assert f(loss=B) == f(counts=A) == f(ws=C) == ga.ERR_OVERLAP

    def b(g=A, gl=B, x=C, counts=D, tokens=D + 64, live=None, t=4, e=8, k=2, ls=8, dt=ga.F32):
        return lib.moe_balance_loss_backward(g, gl, x, counts, tokens, live, t, e, k, ls, dt, 0.1,
                                             None)

    assert b(t=-1) == b(k=0) == ga.ERR_SIZE and b(ls=7) == ga.ERR_STRIDE
    assert b(e=1025, ls=2000) == ga.ERR_TOO_LARGE and b(t=0, g=None) == ga.OK
    for missing in ("g", "gl", "x", "counts", "tokens"):
        assert b(**{missing: None}) == ga.ERR_NULL
    assert b(g=C) == b(g=D) == b(g=B - 4) == ga.ERR_OVERLAP and b(gl=B + 2) == ga.ERR_ALIGN


def test_memory_the_runtime_does_not_know_is_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can run")
    assert _forward(lib, "silu") == ga.ERR_HOST


def test_python_refusals():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    kept = ga.Checkpoint(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ga.silu_and_mul_checkpoint(x)                      # not reachable by the GPU
    with pytest.raises(TypeError):
        ga.silu_and_mul_checkpoint(x.to(torch.int32))
    with pytest.raises(ValueError):
        ga.silu_and_mul_checkpoint(x[0])
    with pytest.raises(ValueError):
        ga.gelu_and_mul_sparse_backward(x, kept, 1.0)      # no std
    with pytest.raises(TypeError):
        ga.checkpoint_values(kept, torch.float16)
    with pytest.raises(ValueError):
        ga.checkpoint_values(ga.Checkpoint(kept.codes[:, :15], kept.scales))
    with pytest.raises(ValueError):
        ga.layer_norm(x, torch.ones(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ga.moe_balance_loss(x, torch.zeros(4, 2, dtype=torch.int64), 0.1)
