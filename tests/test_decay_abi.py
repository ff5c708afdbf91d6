"""Refusals of linear attention with a decay for each head: returned before anything
is enqueued, so these need no GPU; and the reference's own pins."""
import ctypes

import pytest
import torch

import decay_ref as ref
import weight_rnn_gb300 as wr
from block_ref import U
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


def strides(*n):
    return (ctypes.c_int64 * len(n))(*n)


NINE = (2240, 32, 16) * 2 + (1120, 16, 8)
FWD = dict(q=P(1), k=P(2), v=P(3), decay=P(4), h0=None, lengths=None, out=P(5), hT=P(6), B=2, T=70, H=2, dk=16,
           dv=8, strides=NINE, scale=1.0, dtype=1, stream=None)
STEP = dict(q=P(1), k=P(2), v=P(3), decay=P(4), state=P(5), out=P(6), B=2, H=2, dk=16, dv=8,
            strides=(32, 16, 32, 16, 16, 8), scale=1.0, dtype=1, stream=None)
BWD = dict(q=P(1), k=P(2), v=P(3), decay=P(4), h0=None, lengths=None, dout=P(5), dhT=None, dq=P(6), dk_out=P(7),
           dv_out=P(8), dh0=P(9), B=2, T=70, H=2, dk=16, dv=8, strides=NINE, scale=1.0, dtype=1, stream=None)


def call(fn, defaults, kw):
    a = {**defaults, **kw}
    if a["strides"] is not None:
        a["strides"] = strides(*a["strides"])
    return fn(*a.values())


def nine(i, s):
    n = list(NINE)
    n[i] = s
    return dict(strides=tuple(n))


COMMON = [(dict(B=-1), INVALID), (dict(H=-1), INVALID), (dict(dtype=7), INVALID), (dict(dk=0), UNSUP),
          (dict(dv=0), UNSUP), (dict(dk=257), UNSUP), (dict(dv=-3), UNSUP), (dict(strides=None), INVALID),
          (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(decay=None), INVALID),
          (dict(q=P(1, 1)), ALIGN), (dict(k=P(2, 1)), ALIGN), (dict(v=P(3, 1)), ALIGN), (dict(decay=P(4, 2)), ALIGN)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(T=-1), INVALID), (dict(B=1 << 20, T=1 << 20, H=1), UNSUP), (dict(B=1 << 13, H=1 << 12), UNSUP),
    (dict(out=None), INVALID), (nine(0, -8), INVALID), (nine(4, -1), INVALID), (nine(8, 1 << 40), INVALID),
    (dict(lengths=P(8, 2)), ALIGN), (dict(out=P(5, 8)), ALIGN), (dict(hT=P(6, 4)), ALIGN), (dict(h0=P(7, 8)), ALIGN),
    (dict(out=P(1)), INVALID), (dict(out=P(3, 16)), INVALID), (dict(hT=P(5)), INVALID), (dict(hT=P(4)), INVALID),
    (dict(h0=P(6, 16)), INVALID), (dict(h0=P(5)), INVALID),
    (nine(0, 1 << 20) | dict(out=P(1, (1 << 21) + 16)), INVALID),  # inside q's second row
])
def test_fwd_refuses(lib, kw, status):
    assert call(lib.delta_decay_fwd, FWD, kw) == status
    assert wr.delta_last_error() != "no error"


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(state=None), INVALID), (dict(out=None), INVALID), (dict(state=P(5, 4)), ALIGN), (dict(out=P(6, 2)), ALIGN),
    (dict(out=P(5)), INVALID), (dict(state=P(2)), INVALID), (dict(strides=(32, -16, 32, 16, 16, 8)), INVALID),
])
def test_step_refuses(lib, kw, status):
    assert call(lib.delta_decay_step, STEP, kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(T=-1), INVALID), (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(dk_out=None), INVALID),
    (dict(dv_out=None), INVALID), (dict(dout=P(5, 2)), ALIGN), (dict(dq=P(6, 8)), ALIGN), (dict(dh0=P(9, 4)), ALIGN),
    (dict(dhT=P(10, 8)), ALIGN), (dict(dq=P(7)), INVALID), (dict(dv_out=P(5)), INVALID), (dict(dk_out=P(2)), INVALID),
    (dict(dhT=P(9)), INVALID),  # both are at work at once: not in place
    (dict(dhT=P(6)), INVALID), (dict(h0=P(9, 16)), INVALID),
])
def test_bwd_refuses(lib, kw, status):
    assert call(lib.delta_decay_bwd, BWD, kw) == status


def test_nothing_to_do_is_fine(lib):
    for kw in (dict(B=0), dict(H=0), dict(B=0, strides=None, q=None)):
        assert call(lib.delta_decay_fwd, FWD, kw) == wr.DELTA_OK
        assert call(lib.delta_decay_bwd, BWD, kw) == wr.DELTA_OK
        assert call(lib.delta_decay_step, STEP, kw) == wr.DELTA_OK


def test_failure_is_injected(lib):
    for fn, args in ((lib.delta_decay_fwd, FWD), (lib.delta_decay_step, STEP), (lib.delta_decay_bwd, BWD)):
        assert lib.delta_inject_failure(1) == wr.DELTA_OK
        assert call(fn, args, {}) == wr.DELTA_ERR_CUDA
        assert "injected" in wr.delta_last_error()


@pytest.fixture
def python_only(monkeypatch):
    monkeypatch.setattr(block, "_lib", lambda: pytest.fail("the library was reached"))
    monkeypatch.setattr(block, "_fast", block._Nothing())


def fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return Fake(*shape, dtype=dtype, device=device)


def good():
    return dict(q=fake(2, 5, 3, 16), k=fake(2, 5, 3, 16), v=fake(2, 5, 3, 8), decay=fake(3, dtype=F32))


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(2, 5, 3, 16)), ValueError), (dict(q=fake(2, 5, 16)), ValueError), (dict(q=None), TypeError),
    (dict(q=fake(2, 5, 3, 16, dtype=torch.float16)), TypeError), (dict(k=fake(2, 5, 2, 16)), ValueError),
    (dict(k=fake(2, 5, 3, 16, dtype=F32)), TypeError), (dict(k=None), TypeError), (dict(v=fake(2, 4, 3, 8)), ValueError),
    (dict(v=None), ValueError), (dict(decay=fake(2, dtype=F32)), ValueError), (dict(decay=fake(3)), TypeError),
    (dict(decay=fake(3, dtype=F32, device="cuda:1")), ValueError), (dict(h0=fake(2, 3, 16, 16, dtype=F32)), ValueError),
    (dict(h0=fake(2, 3, 16, 8)), TypeError), (dict(lengths=fake(2, dtype=torch.int64)), TypeError),
    (dict(lengths=fake(3, dtype=torch.int32)), ValueError), (dict(v=fake(2, 5, 3, 1 << 32)), ValueError),
    (dict(q=fake(1 << 32, 5, 3, 16)), ValueError),
])
def test_python_refuses(python_only, kw, error):
    a = {**good(), **kw}
    with pytest.raises(error):
        wr.delta_decay_fwd(**a)
    with pytest.raises(error):
        wr.delta_decay_bwd(**a, dout=fake(2, 5, 3, 8))


def test_python_refuses_a_steps_state(python_only):
    a = dict(q=fake(2, 3, 16), k=fake(2, 3, 16), v=fake(2, 3, 8), decay=fake(3, dtype=F32))
    for state, error in ((fake(2, 3, 8, 16, dtype=F32), ValueError), (fake(2, 3, 16, 8), TypeError), (None, TypeError)):
        with pytest.raises(error):
            wr.delta_decay_step(**a, state=state)
    with pytest.raises(ValueError):
        wr.delta_decay_step(**{**a, "v": fake(2, 3, 3, 8)}, state=fake(2, 3, 16, 8, dtype=F32))


# ------------------------------------------------------------------ the reference
def test_reference_equals_the_closed_form():
    """sum over j <= t of g^(t-j) (q_t k_j) v_j + g^(t+1) q_t h0"""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, 9, 3, d, generator=gen) for d in (4, 4, 5))
    decay, h0 = torch.tensor([0.0, 1.0, 0.7]), torch.randn(2, 3, 4, 5, generator=gen)
    out, hT, _, _ = ref.forward(q, k, v, decay, h0, 0.5, torch.tensor([9, 4]))
    for b, n in enumerate((9, 4)):
        for h, g in enumerate(decay.double().tolist()):
            d = lambda t: t[b, :n, h].double()  # noqa: E731
            i = torch.arange(n)
            w = torch.where(i[:, None] >= i, g ** (i[:, None] - i).clamp(min=0).double(), 0.0)
            want = (d(q) @ d(k).T * w) @ d(v) + g ** (i[:, None] + 1.0) * (d(q) @ h0[b, h].double())
            torch.testing.assert_close(out[b, :n, h], 0.5 * want)
        assert not out[b, n:].any()


def test_reference_gradients_are_autograds():
    gen = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(1, 7, 2, d, generator=gen, dtype=torch.float64, requires_grad=True) for d in (3, 3, 4))
    h0 = torch.randn(1, 2, 3, 4, generator=gen, dtype=torch.float64, requires_grad=True)
    decay = torch.tensor([0.3, 0.95])
    do, dh = torch.randn(1, 7, 2, 4, generator=gen), torch.randn(1, 2, 3, 4, generator=gen)
    S, loss = h0[0], 0.0
    for t in range(5):
        S = decay.double()[:, None, None] * S + k[0, t][..., None] * v[0, t][:, None]
        loss = loss + (2.0 * (q[0, t][:, None] @ S)[:, 0] * do[0, t]).sum()
    loss = loss + (S * dh[0]).sum()
    want = torch.autograd.grad(loss, (q, k, v, h0))
    got, big = ref.backward(q.detach(), k.detach(), v.detach(), decay, do, h0.detach(), dh, 2.0, torch.tensor([5]))
    for g, w, m in zip(got, want, big):
        torch.testing.assert_close(g, w)
        assert (g.abs() <= m * (1 + 100 * U)).all()
