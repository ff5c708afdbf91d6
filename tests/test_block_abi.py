"""Refusals of the block operators: every argument error is returned before
anything is enqueued, so these need no GPU."""
import ctypes

import pytest
import torch

import weight_rnn_gb300 as wr
from weight_rnn_gb300 import build as wbuild

INVALID, UNSUP, ALIGN = wr.DELTA_ERR_INVALID, wr.DELTA_ERR_UNSUPPORTED, wr.DELTA_ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return wr.load_library()


def P(i, off=0):  # pointers 2^40 apart: aligned, never dereferenced
    return (i << 40) + off


def call(fn, order, defaults, kw):
    a = {**defaults, **kw}
    return fn(*(a[n] for n in order))


SCAN = dict(x=P(1), gate=P(2), h0=None, lengths=None, out=P(3), hT=P(4), states=None, B=2, T=70, D=8,
            x_sb=560, x_st=8, g_sb=560, g_st=8, dtype=1, form=1, stream=None)
STEP = dict(x=P(1), gate=P(2), state=P(3), out=P(4), B=2, D=8, x_sb=8, g_sb=8, dtype=1, form=1, stream=None)
SBWD = dict(x=P(1), gate=P(2), states=P(3), lengths=None, dout=P(4), dhT=None, dx=P(5), dgate=P(6),
            dh0=P(7), B=2, T=70, D=8, x_sb=560, x_st=8, g_sb=560, g_st=8, dtype=1, form=1, stream=None)
NORM = dict(x=P(1), residual=P(2), weight=P(3), y=P(4), sum_out=P(5), rstd=P(6), rows=4, D=64, ldx=64,
            ldr=64, eps=1e-6, dtype=1, wdtype=0, stream=None)
QUANT = dict(x=P(1), residual=P(2), weight=P(3), y=P(4), y_scale=P(5), sum_out=P(6), rows=4, D=64, ldx=64,
             ldr=64, eps=1e-6, dtype=1, wdtype=0, stream=None)
NBWD = dict(dy=P(1), sum=P(2), weight=P(3), rstd=P(4), dsum=None, dx=P(5), dweight=P(6), rows=4, D=64,
            dtype=1, wdtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-1), INVALID),
    (dict(dtype=7), INVALID), (dict(form=2), INVALID),
    (dict(x=None), INVALID), (dict(gate=None), INVALID), (dict(out=None), INVALID),
    (dict(x_sb=-8), INVALID), (dict(g_st=-1), INVALID), (dict(x_st=1 << 41), INVALID),
    (dict(x_st=1 << 39), UNSUP), (dict(B=1 << 30, D=1 << 12), UNSUP),
    (dict(B=1 << 20, T=1 << 20, D=8), UNSUP),
    (dict(x=P(1, 1)), ALIGN), (dict(gate=P(2, 1)), ALIGN), (dict(lengths=P(8, 2)), ALIGN),
    (dict(form=0, gate=P(2, 2)), ALIGN), (dict(out=P(3, 8)), ALIGN), (dict(hT=P(4, 4)), ALIGN),
    (dict(states=P(9, 4)), ALIGN), (dict(h0=P(9, 2)), ALIGN),
    (dict(out=P(1)), INVALID), (dict(out=P(2, 16)), INVALID), (dict(states=P(3, 32)), INVALID),
    (dict(hT=P(3)), INVALID), (dict(h0=P(9), hT=P(9, 16)), INVALID), (dict(h0=P(3)), INVALID),
    # the view reaches past its first row: out lies inside it
    (dict(x_sb=1 << 20, out=P(1, (1 << 21) + 64)), INVALID),
])
def test_scan_fwd_refuses(lib, kw, status):
    assert call(lib.delta_scan_fwd, SCAN, SCAN, kw) == status
    assert wr.delta_last_error() != "no error"


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(D=-1), INVALID), (dict(dtype=2), INVALID), (dict(form=-1), INVALID),
    (dict(state=None), INVALID), (dict(out=None), INVALID), (dict(x=None), INVALID),
    (dict(x_sb=-1), INVALID), (dict(state=P(3, 4)), ALIGN), (dict(out=P(4, 2)), ALIGN),
    (dict(x=P(1, 1)), ALIGN), (dict(out=P(3)), INVALID), (dict(state=P(1)), INVALID),
])
def test_scan_step_refuses(lib, kw, status):
    assert call(lib.delta_scan_step, STEP, STEP, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(dtype=9), INVALID), (dict(form=5), INVALID),
    (dict(states=None), INVALID), (dict(dout=None), INVALID), (dict(dx=None), INVALID),
    (dict(dgate=None), INVALID), (dict(x=None), INVALID),
    (dict(dout=P(4, 2)), ALIGN), (dict(dx=P(5, 8)), ALIGN), (dict(states=P(3, 4)), ALIGN),
    (dict(dh0=P(7, 4)), ALIGN), (dict(gate=P(2, 1)), ALIGN),
    (dict(dx=P(4)), INVALID), (dict(dgate=P(5)), INVALID), (dict(dx=P(1)), INVALID),
    (dict(dh0=P(3)), INVALID), (dict(dhT=P(8), dh0=P(8, 16)), INVALID), (dict(dhT=P(5)), INVALID),
])
def test_scan_bwd_refuses(lib, kw, status):
    assert call(lib.delta_scan_bwd, SBWD, SBWD, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(D=-1), INVALID), (dict(dtype=2), INVALID), (dict(wdtype=3), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(D=8193, ldx=8193, ldr=8193), UNSUP), (dict(rows=1 << 40), UNSUP),
    (dict(ldx=63), INVALID), (dict(ldr=0), INVALID), (dict(ldx=1 << 40), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(residual=None), INVALID),  # a sum to write, but no residual
    (dict(x=P(1, 1)), ALIGN), (dict(weight=P(3, 2)), ALIGN), (dict(y=P(4, 2)), ALIGN),
    (dict(sum_out=P(5, 8)), ALIGN), (dict(rstd=P(6, 4)), ALIGN),
    (dict(y=P(1)), INVALID), (dict(y=P(2)), INVALID), (dict(rstd=P(3)), INVALID),
    (dict(sum_out=P(4)), INVALID), (dict(sum_out=P(2, 128)), INVALID),
    (dict(sum_out=P(2), ldr=128), INVALID),  # in place, but the rows lie elsewhere
])
def test_norm_fwd_refuses(lib, kw, status):
    assert call(lib.delta_add_rmsnorm_fwd, NORM, NORM, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y_scale=None), INVALID), (dict(eps=0.0), INVALID), (dict(y=P(4, 1)), ALIGN),
    (dict(y_scale=P(5, 4)), ALIGN), (dict(y_scale=P(4)), INVALID), (dict(sum_out=P(4, 16)), INVALID),
])
def test_norm_quant_refuses(lib, kw, status):
    assert call(lib.delta_add_rmsnorm_quant, QUANT, QUANT, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(dtype=2), INVALID), (dict(D=9000), UNSUP),
    (dict(dy=None), INVALID), (dict(sum=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(weight=None), INVALID), (dict(dweight=None), INVALID),
    (dict(dy=P(1, 2)), ALIGN), (dict(dsum=P(7, 8)), ALIGN), (dict(dweight=P(6, 4)), ALIGN),
    (dict(dx=P(2)), INVALID), (dict(dx=P(1, 64)), INVALID), (dict(dweight=P(1)), INVALID),
    (dict(dweight=P(5)), INVALID),
])
def test_norm_bwd_refuses(lib, kw, status):
    assert call(lib.delta_add_rmsnorm_bwd, NBWD, NBWD, kw) == status

LIN = dict(x=P(1), w=P(2), bias=P(3), residual=P(4), out=P(5), pre=P(6), M=40, N=64, K=32, ldx=32, ldw=32,
           ldr=64, act=1, dtype=1, bdtype=0, stream=None)
LQ = dict(x=P(1), x_scale=P(2), w=P(3), w_scale=P(4), bias=P(5), residual=P(6), out=P(7), M=40, N=64, K=32,
          ldx=32, ldw=32, ldr=64, act=1, bdtype=0, stream=None)
LB = dict(x=P(1), w=P(2), dout=P(3), pre=P(4), dx=P(5), dw=P(6), dbias=P(7), M=40, N=64, K=32, ldx=32,
          ldw=32, act=1, dtype=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(K=0), INVALID),
    (dict(act=3), INVALID), (dict(dtype=2), INVALID), (dict(bdtype=5), INVALID),
    (dict(ldx=31), INVALID), (dict(ldw=31), INVALID), (dict(ldr=63), INVALID), (dict(ldx=1 << 31), UNSUP),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P(1, 1)), ALIGN), (dict(w=P(2, 1)), ALIGN), (dict(bias=P(3, 2)), ALIGN),
    (dict(residual=P(4, 1)), ALIGN), (dict(out=P(5, 8)), ALIGN), (dict(pre=P(6, 2)), ALIGN),
    (dict(out=P(1)), INVALID), (dict(out=P(2, 32)), INVALID), (dict(out=P(3)), INVALID),
    (dict(out=P(4, 128)), INVALID), (dict(out=P(4), ldr=72), INVALID), (dict(pre=P(4)), INVALID),
    (dict(pre=P(5)), INVALID),
])
def test_linear_fwd_refuses(lib, kw, status):
    assert call(lib.delta_linear_fwd, LIN, LIN, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), INVALID), (dict(act=-1), INVALID), (dict(x_scale=None), INVALID), (dict(w_scale=None), INVALID),
    (dict(x_scale=P(2, 2)), ALIGN), (dict(w_scale=P(4, 1)), ALIGN), (dict(out=P(7, 4)), ALIGN),
    (dict(out=P(2)), INVALID), (dict(out=P(4)), INVALID), (dict(residual=P(6, 1)), ALIGN),
])
def test_linear_quant_refuses(lib, kw, status):
    assert call(lib.delta_linear_quant, LQ, LQ, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(act=9), INVALID), (dict(dtype=2), INVALID),
    (dict(dout=None), INVALID), (dict(pre=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(ldx=8), INVALID), (dict(ldw=8), INVALID),
    (dict(dout=P(3, 2)), ALIGN), (dict(pre=P(4, 8)), ALIGN), (dict(dx=P(5, 2)), ALIGN),
    (dict(dbias=P(7, 4)), ALIGN), (dict(x=P(1, 1)), ALIGN),
    (dict(dx=P(1)), INVALID), (dict(dw=P(2)), INVALID), (dict(dw=P(3)), INVALID), (dict(dbias=P(4)), INVALID),
    (dict(dw=P(5)), INVALID),
])
def test_linear_bwd_refuses(lib, kw, status):
    assert call(lib.delta_linear_bwd, LB, LB, kw) == status


def test_empty_problems_are_fine(lib):
    assert call(lib.delta_linear_fwd, LIN, LIN, dict(M=0)) == 0
    assert call(lib.delta_linear_quant, LQ, LQ, dict(N=0)) == 0
    assert call(lib.delta_linear_bwd, LB, LB, dict(dx=None, dw=None, dbias=None)) == 0
    assert call(lib.delta_scan_fwd, SCAN, SCAN, dict(B=0)) == 0
    assert call(lib.delta_scan_fwd, SCAN, SCAN, dict(D=0)) == 0
    assert call(lib.delta_scan_step, STEP, STEP, dict(B=0)) == 0
    assert call(lib.delta_scan_bwd, SBWD, SBWD, dict(B=0)) == 0
    assert call(lib.delta_add_rmsnorm_fwd, NORM, NORM, dict(rows=0)) == 0
    assert call(lib.delta_add_rmsnorm_bwd, NBWD, NBWD, dict(D=0)) == 0


@pytest.mark.parametrize("name,order", [
    ("delta_scan_fwd", SCAN), ("delta_scan_step", STEP), ("delta_scan_bwd", SBWD),
    ("delta_add_rmsnorm_fwd", NORM), ("delta_add_rmsnorm_quant", QUANT), ("delta_add_rmsnorm_bwd", NBWD),
    ("delta_linear_fwd", LIN), ("delta_linear_quant", LQ), ("delta_linear_bwd", LB)])
def test_injected_failure(lib, name, order):
    wr.delta_inject_failure(1)
    try:
        assert getattr(lib, name)(*order.values()) == wr.DELTA_ERR_CUDA
        assert "injected" in wr.delta_last_error()
    finally:
        wr.delta_inject_failure(0)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(1, 4, 8), torch.ones(8)
    for f in (lambda: wr.delta_scan_fwd(x, x), lambda: wr.delta_scan_step(x[0], x[0], x[0]),
              lambda: wr.delta_scan_bwd(x, x, x, x), lambda: wr.delta_add_rmsnorm_fwd(x, w),
              lambda: wr.delta_linear_fwd(x, x[0]), lambda: wr.delta_linear_bwd(x, x[0], x),
              lambda: wr.delta_linear_quant(x, w, x[0], w), lambda: wr.delta_add_rmsnorm_quant(x, w), lambda: wr.delta_add_rmsnorm_bwd(x, x, w, x[..., 0])):
        with pytest.raises(ValueError, match="needs CUDA tensors"):
            f()


def test_binding_checks_types_and_forms():
    with pytest.raises(TypeError):
        wr.delta_scan_fwd("x", None)
    with pytest.raises(TypeError):
        wr.delta_add_rmsnorm_fwd(None, None)
