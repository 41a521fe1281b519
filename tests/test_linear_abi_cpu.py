"""Refusals of the gated projections and the cross entropy: sizes, strides, types, pointers,
workspaces.  No call here launches a kernel: each fails its checks before any CUDA call, or has
nothing to do."""
import ctypes

import pytest

import gated_activation_gb300 as ga
from gated_activation_gb300 import build as gbuild

A, B, C, D, E, F, G, W = (0x100000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    if not gbuild.up_to_date():
        gbuild.build()
    return ga.load_library()


def _operands(x=A, w=B, e=1, t=4, k=16, d=8, xs=16, xb=0, ws=16, wb=0, dtype=ga.BF16, n=None):
    return ctypes.byref(ga.LinearOperands(x, w, e, t, k, d, xs, xb, ws, wb, dtype, n))


def _vocabulary(x=A, w=B, goal=C, t=4, k=16, v=32, xs=16, ws=16, dtype=ga.BF16, wide=1):
    return ctypes.byref(ga.VocabularyOperands(x, w, goal, t, k, v, xs, ws, dtype, wide))


@pytest.mark.parametrize("name", ["linear_silu_and_mul", "linear_gelu_and_mul"])
def test_forward_refusals(lib, name):
    def f(out=D, codes=None, scales=None, work=W, size=1 << 30, **a):
        return getattr(lib, name)(out, codes, scales, _operands(**a), work, size, None)

    assert getattr(lib, name)(D, None, None, None, W, 0, None) == ga.ERR_NULL
    assert f(t=-1) == f(e=-1) == f(d=0) == f(k=0) == f(d=-3) == ga.ERR_SIZE
    assert f(dtype=ga.F32) == f(dtype=7) == ga.ERR_DTYPE
    assert f(xs=15) == f(ws=15) == f(e=2, xb=63, wb=256) == f(e=2, xb=64, wb=255) == ga.ERR_STRIDE
    assert f(e=1025, xb=64, wb=256) == f(d=1 << 31, ws=16) == f(t=1 << 31) == f(k=1 << 31, xs=1 << 32, ws=1 << 32) \
        == f(t=1 << 30, d=1 << 30) == f(xs=1 << 41) == ga.ERR_TOO_LARGE
    assert f(t=0, x=None, out=None) == f(e=0, x=None, w=None, out=None) == ga.OK
    assert f(x=None) == f(w=None) == f(out=None) == f(codes=E) == f(scales=F) == ga.ERR_NULL
    assert f(x=A + 1) == f(out=D + 1) == f(codes=E + 1, scales=F) == f(n=G + 2) == ga.ERR_ALIGN
    # out spans 64 bytes, codes 128, scales 8, in 128, weight 512
    assert f(out=A) == f(out=A + 126) == f(out=B + 510) == f(codes=D + 62, scales=F) \
        == f(codes=E, scales=E + 127) == f(n=D) == ga.ERR_OVERLAP


def test_forward_workspace(lib):
    def need(**a):
        return lib.linear_and_mul_workspace_bytes(_operands(**a))

    assert need() == need(x=A + 16, xs=24) == need(t=0) == need(t=-1) == 0
    # rows that 16-byte copies cannot read: padded copies of 4 x 16 and of 16 x 16 elements
    assert need(x=A + 2) == 128 and need(w=B + 2) == 512 and need(xs=17, ws=17) == 640
    assert need(k=15) == 0 and need(k=15, xs=15, ws=15) == 640
    f = lambda work, size, **a: lib.linear_silu_and_mul(D, E, F, _operands(**a), work, size, None)  # noqa: E731
    assert f(W, 639, xs=17, ws=17) == ga.ERR_SCRATCH
    assert f(None, 640, xs=17, ws=17) == ga.ERR_NULL
    assert f(W + 8, 640, xs=17, ws=17) == ga.ERR_ALIGN and f(A, 640, xs=17, ws=17) == ga.ERR_OVERLAP


@pytest.mark.parametrize("name", ["linear_silu_and_mul_backward", "linear_gelu_and_mul_backward"])
def test_backward_refusals(lib, name):
    def f(gi=D, gw=E, dy=F, gs=8, gb=0, codes=G, scales=G + 4096, work=W, size=1 << 30, **a):
        return getattr(lib, name)(gi, gw, dy, gs, gb, codes, scales, _operands(**a), work, size, None)

    assert getattr(lib, name)(D, E, F, 8, 0, G, G + 4096, None, W, 0, None) == ga.ERR_NULL
    assert f(t=-1) == f(d=0) == f(k=0) == ga.ERR_SIZE and f(dtype=ga.F32) == ga.ERR_DTYPE
    assert f(gs=7) == f(xs=15) == f(e=2, xb=64, wb=256, gb=31) == ga.ERR_STRIDE
    assert f(gs=1 << 41) == f(t=1 << 31) == ga.ERR_TOO_LARGE
    assert f(e=0) == ga.OK
    need = lib.linear_and_mul_backward_workspace_bytes(_operands())
    assert need == 2 * 64 * 8 * 2                # dg and du, whole steps of 64 rows
    assert lib.linear_and_mul_backward_workspace_bytes(_operands(n=G)) == need + 64 * 16 * 2
    assert f(size=need - 1) == ga.ERR_SCRATCH
    for missing in ("gi", "gw", "dy", "codes", "scales", "work", "x", "w"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(gi=D + 1) == f(dy=F + 1) == f(codes=G + 1) == f(work=W + 8) == ga.ERR_ALIGN
    assert f(gi=A) == f(gw=B) == f(gw=D + 126) == f(gi=F) == f(gw=G) == f(work=A) == ga.ERR_OVERLAP


def test_entropy_refusals(lib):
    def f(loss=D, lse=E, work=W, size=1 << 30, **a):
        return lib.linear_cross_entropy(loss, lse, _vocabulary(**a), work, size, None)

    assert lib.linear_cross_entropy(D, E, None, W, 0, None) == ga.ERR_NULL
    assert f(t=-1) == f(k=0) == f(v=0) == ga.ERR_SIZE and f(dtype=ga.F32) == ga.ERR_DTYPE
    assert f(xs=15) == f(ws=15) == ga.ERR_STRIDE
    assert f(t=1 << 31) == f(v=1 << 31) == f(t=1 << 30, v=1 << 30) == ga.ERR_TOO_LARGE
    assert f(t=0, x=None, loss=None) == ga.OK
    need = lib.linear_cross_entropy_workspace_bytes(_vocabulary())
    assert need > 0 and f(size=need - 1) == ga.ERR_SCRATCH
    for missing in ("loss", "lse", "x", "w", "goal", "work"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(loss=D + 2) == f(goal=C + 4) == f(x=A + 1) == ga.ERR_ALIGN
    assert f(loss=A) == f(lse=D + 12) == f(loss=C) == f(work=B) == ga.ERR_OVERLAP


def test_entropy_backward_refusals(lib):
    def f(gi=D, gw=E, gl=F, loss=F + 4096, lse=G, work=W, size=1 << 30, **a):
        return lib.linear_cross_entropy_backward(gi, gw, gl, loss, lse, _vocabulary(**a), work, size, None)

    assert lib.linear_cross_entropy_backward(D, E, F, F + 4096, G, None, W, 0, None) == ga.ERR_NULL
    assert f(t=-1) == f(v=-1) == ga.ERR_SIZE and f(dtype=ga.F32) == ga.ERR_DTYPE
    need = lib.linear_cross_entropy_backward_workspace_bytes(_vocabulary())
    assert need > 0 and f(size=need - 1) == ga.ERR_SCRATCH
    # rows off 16-byte boundaries: the weight's copy is added, 32 padded rows
    assert lib.linear_cross_entropy_backward_workspace_bytes(_vocabulary(w=B + 2)) == need + 32 * 16 * 2
    for missing in ("gi", "gw", "gl", "loss", "lse", "x", "w", "goal", "work"):
        assert f(**{missing: None}) == ga.ERR_NULL
    assert f(gi=D + 1) == f(gl=F + 2) == f(goal=C + 2, wide=0) == ga.ERR_ALIGN
    assert f(gi=A) == f(gw=B) == f(gw=F) == f(gi=G) == f(gi=C) == f(gi=F + 4096) == ga.ERR_OVERLAP
