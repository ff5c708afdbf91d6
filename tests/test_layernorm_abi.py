"""Refusals of layer norm: returned before anything is enqueued, so these need no GPU."""
import pytest
import torch

import weight_rnn_gb300 as wr
from fakes import Fake
from weight_rnn_gb300 import block
from weight_rnn_gb300 import build as wbuild

INVALID, UNSUP, ALIGN = wr.DELTA_ERR_INVALID, wr.DELTA_ERR_UNSUPPORTED, wr.DELTA_ERR_ALIGN
F32 = torch.float32


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return wr.load_library()


def P(i, off=0):  # pointers 2^40 apart: aligned, never dereferenced
    return (i << 40) + off


FWD = dict(x=P(1), residual=P(2), weight=P(3), bias=P(4), y=P(5), sum_out=P(6), mean=P(7), rstd=P(8), rows=4, D=64,
           ldx=64, ldr=64, eps=1e-5, dtype=1, wdtype=0, bdtype=1, stream=None)
BWD = dict(dy=P(1), sum=P(2), weight=P(3), mean=P(4), rstd=P(5), dsum=None, dx=P(6), dweight=P(7), dbias=P(8), rows=4,
           D=64, dtype=1, wdtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(D=-1), INVALID), (dict(dtype=2), INVALID), (dict(wdtype=3), INVALID),
    (dict(bdtype=3), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(D=8193, ldx=8193, ldr=8193), UNSUP), (dict(ldx=63), INVALID), (dict(ldr=0), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(residual=None), INVALID),
    (dict(x=P(1, 1)), ALIGN), (dict(weight=P(3, 2)), ALIGN), (dict(bias=P(4, 1)), ALIGN),
    (dict(bias=P(4, 2), bdtype=0), ALIGN), (dict(y=P(5, 2)), ALIGN), (dict(mean=P(7, 4)), ALIGN),
    (dict(rstd=P(8, 4)), ALIGN), (dict(sum_out=P(6, 8)), ALIGN),
    (dict(y=P(1)), INVALID), (dict(y=P(4)), INVALID), (dict(mean=P(8)), INVALID), (dict(mean=P(4)), INVALID),
    (dict(mean=P(5)), INVALID), (dict(sum_out=P(7)), INVALID), (dict(sum_out=P(4)), INVALID),
    (dict(sum_out=P(2, 128)), INVALID), (dict(sum_out=P(2), ldr=128), INVALID),
])
def test_fwd_refuses(lib, kw, status):
    assert lib.delta_add_layernorm_fwd(*{**FWD, **kw}.values()) == status
    assert wr.delta_last_error() != "no error"


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(dtype=2), INVALID), (dict(D=9000), UNSUP), (dict(dy=None), INVALID),
    (dict(sum=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID),
    (dict(weight=None), INVALID), (dict(dweight=None), INVALID), (dict(dbias=None), INVALID),
    (dict(dy=P(1, 2)), ALIGN), (dict(mean=P(4, 4)), ALIGN), (dict(dbias=P(8, 4)), ALIGN), (dict(dsum=P(9, 8)), ALIGN),
    (dict(dx=P(2)), INVALID), (dict(dx=P(1, 64)), INVALID), (dict(dbias=P(7)), INVALID), (dict(dbias=P(4)), INVALID),
    (dict(dweight=P(6)), INVALID), (dict(dbias=P(1)), INVALID),
])
def test_bwd_refuses(lib, kw, status):
    assert lib.delta_add_layernorm_bwd(*{**BWD, **kw}.values()) == status


def test_failure_is_injected(lib):
    for fn, args in ((lib.delta_add_layernorm_fwd, FWD), (lib.delta_add_layernorm_bwd, BWD)):
        assert lib.delta_inject_failure(1) == wr.DELTA_OK
        assert fn(*args.values()) == wr.DELTA_ERR_CUDA


def fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return Fake(*shape, dtype=dtype, device=device)


@pytest.mark.parametrize("kw,error", [
    (dict(x=torch.zeros(2, 8)), ValueError), (dict(x=None), TypeError), (dict(weight=None), TypeError),
    (dict(weight=fake(9)), ValueError), (dict(bias=fake(9)), ValueError), (dict(bias=fake(8, dtype=torch.float16)), TypeError),
    (dict(bias=fake(8, device="cuda:1")), ValueError), (dict(residual=fake(3, 8)), ValueError),
    (dict(x=fake(2, (1 << 32) + 8)), ValueError), (dict(sum_out=fake(2, 8)), ValueError),
])
def test_python_refuses(monkeypatch, kw, error):
    monkeypatch.setattr(block, "_lib", lambda: pytest.fail("the library was reached"))
    monkeypatch.setattr(block, "_fast", block._Nothing())
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Fake(1))
    with pytest.raises(error):
        wr.delta_add_layernorm_fwd(**{**dict(x=fake(2, 8), weight=fake(8, dtype=F32)), **kw})


@pytest.mark.parametrize("kw,error", [
    (dict(mean=fake(3, dtype=F32)), ValueError), (dict(mean=fake(2)), TypeError), (dict(mean=None), TypeError),
    (dict(sum=fake(2, 8, dtype=F32)), TypeError), (dict(dsum=fake(2, 9)), ValueError),
])
def test_python_refuses_for_gradients(monkeypatch, kw, error):
    monkeypatch.setattr(block, "_lib", lambda: pytest.fail("the library was reached"))
    monkeypatch.setattr(block, "_fast", block._Nothing())
    good = dict(dy=fake(2, 8), sum=fake(2, 8), weight=fake(8), mean=fake(2, dtype=F32), rstd=fake(2, dtype=F32))
    with pytest.raises(error):
        wr.delta_add_layernorm_bwd(**{**good, **kw})
