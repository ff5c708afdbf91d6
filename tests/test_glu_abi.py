"""Refusals of the gated layer: returned before anything is enqueued, so these need
no GPU."""
import pytest
import torch

import weight_rnn_gb300 as wr
from fakes import Fake, Library
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


FWD = dict(x=P(1), w=P(2), bias=P(3), out=P(4), pre=P(5), M=4, N=8, K=16, ldx=16, ldw=16, act=1, dtype=1, bdtype=0,
           stream=None)
BWD = dict(x=P(1), w=P(2), dout=P(3), pre=P(4), dx=P(5), dw=P(6), dbias=P(7), M=4, N=8, K=16, ldx=16, ldw=16, act=1,
           dtype=1, stream=None)

COMMON = [(dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(K=0), INVALID),
          (dict(N=(1 << 30) + 1), UNSUP), (dict(N=1 << 30), UNSUP), (dict(act=3), INVALID), (dict(dtype=2), INVALID), (dict(ldx=15), INVALID),
          (dict(ldw=15), INVALID), (dict(N=1, ldw=8), INVALID), (dict(ldw=1 << 31), UNSUP),
          (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=P(1, 1)), ALIGN), (dict(w=P(2, 1)), ALIGN)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(bdtype=5), INVALID), (dict(out=None), INVALID), (dict(bias=P(3, 2)), ALIGN), (dict(out=P(4, 8)), ALIGN),
    (dict(pre=P(5, 2)), ALIGN), (dict(out=P(1)), INVALID), (dict(out=P(2, 256)), INVALID),  # w's second half
    (dict(pre=P(3)), INVALID), (dict(pre=P(4)), INVALID),
])
def test_fwd_refuses(lib, kw, status):
    assert lib.delta_glu_fwd(*{**FWD, **kw}.values()) == status
    assert wr.delta_last_error() != "no error"


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dout=None), INVALID), (dict(pre=None), INVALID), (dict(pre=None, act=0), INVALID), (dict(dout=P(3, 2)), ALIGN),
    (dict(dx=P(5, 8)), ALIGN), (dict(dw=P(6, 2)), ALIGN), (dict(dbias=P(7, 4)), ALIGN), (dict(dx=P(3)), INVALID),
    (dict(dw=P(2)), INVALID), (dict(dbias=P(6)), INVALID), (dict(dx=P(4, 64)), INVALID),
])
def test_bwd_refuses(lib, kw, status):
    assert lib.delta_glu_bwd(*{**BWD, **kw}.values()) == status


def test_failure_is_injected_and_nothing_to_do_is_fine(lib):
    for fn, args in ((lib.delta_glu_fwd, FWD), (lib.delta_glu_bwd, BWD)):
        assert lib.delta_inject_failure(1) == wr.DELTA_OK
        assert fn(*args.values()) == wr.DELTA_ERR_CUDA
    assert lib.delta_glu_fwd(*{**FWD, "M": 0}.values()) == wr.DELTA_OK
    assert lib.delta_glu_bwd(*{**BWD, "dx": None, "dw": None, "dbias": None}.values()) == wr.DELTA_OK


def fake(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return Fake(*shape, dtype=dtype, device=device)


@pytest.fixture
def python_only(monkeypatch):
    monkeypatch.setattr(block, "_lib", lambda: pytest.fail("the library was reached"))
    monkeypatch.setattr(block, "_fast", block._Nothing())


@pytest.mark.parametrize("kw,error", [
    (dict(x=torch.zeros(2, 8)), ValueError), (dict(x=None), TypeError), (dict(w=fake(7, 8)), ValueError),
    (dict(w=fake(6, 9)), ValueError), (dict(w=None), ValueError), (dict(w=fake(6, 8, dtype=F32)), TypeError),
    (dict(act="relu"), ValueError), (dict(x=fake(1 << 32, 8)), ValueError), (dict(x=fake(2, 8, device="cuda:1")), ValueError),
])
def test_python_refuses(python_only, kw, error):
    a = {**dict(x=fake(2, 8), w=fake(6, 8)), **kw}
    with pytest.raises(error):
        wr.delta_glu_fwd(**a)
    with pytest.raises(error):
        wr.delta_glu_bwd(**a, dout=fake(2, 3), pre=fake(2, 6))


def test_python_refuses_the_rest(python_only):
    x, w = fake(2, 8), fake(6, 8)
    for bias, error in ((fake(3), ValueError), (fake(6, dtype=torch.float16), TypeError)):
        with pytest.raises(error):
            wr.delta_glu_fwd(x, w, bias)
    with pytest.raises(ValueError):
        wr.delta_glu_fwd(x, w, out=fake(2, 6))
    for dout, pre, error in ((fake(2, 6), fake(2, 6), ValueError), (fake(2, 3), fake(2, 3), ValueError),
                             (fake(2, 3), None, TypeError), (fake(2, 3, dtype=F32), fake(2, 6), TypeError)):
        with pytest.raises(error):
            wr.delta_glu_bwd(x, w, dout, pre)


# ---- the newer calls on a device that is not the current one
def made(device):
    t = lambda *s, dtype=torch.bfloat16: Fake(*s, dtype=dtype, device=device)  # noqa: E731
    f = lambda *s: t(*s, dtype=F32)  # noqa: E731
    x, q, s = t(2, 8), t(1, 4, 2, 16), f(1, 2, 16, 16)
    return {
        "delta_glu_fwd": lambda: wr.delta_glu_fwd(x, t(6, 8), f(6)),
        "delta_glu_bwd": lambda: wr.delta_glu_bwd(x, t(6, 8), t(2, 3), t(2, 6)),
        "delta_add_layernorm_fwd": lambda: wr.delta_add_layernorm_fwd(x, t(8), t(8), x),
        "delta_add_layernorm_bwd": lambda: wr.delta_add_layernorm_bwd(x, x, t(8), f(2), f(2)),
        "delta_decay_fwd": lambda: wr.delta_decay_fwd(q, q, q, f(2), s),
        "delta_decay_bwd": lambda: wr.delta_decay_bwd(q, q, q, f(2), q, s, s),
        "delta_decay_step": lambda: wr.delta_decay_step(t(1, 2, 16), t(1, 2, 16), t(1, 2, 16), f(2), s),
    }


@pytest.mark.parametrize("name", made("cuda:0"))
@pytest.mark.parametrize("index", [0, 1])
def test_library_sees_the_tensors_device(monkeypatch, name, index):
    now, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.index = dev.index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    lib = Library(lambda name, args: seen.append((name, now[0])))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(block, "_current_device", lambda: now[0], raising=False)
    monkeypatch.setattr(block, "_lib", lambda: lib)
    monkeypatch.setattr(block, "_fast", block._Nothing())
    monkeypatch.setattr(block, "_current", lambda index: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, dtype=None, device=None: Fake(
        *(a[0] if len(a) == 1 else a), dtype=dtype, device=device))
    made(f"cuda:{index}")[name]()
    assert seen == [(name, index)] and now == [0]
