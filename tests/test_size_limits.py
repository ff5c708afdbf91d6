"""Sizes that no C int holds are refused by the Python calls, before anything is
allocated or passed on."""
import pytest
import torch

import weight_rnn_gb300 as wr
from fakes import Fake, Library
from weight_rnn_gb300 import block

BIG = (1 << 32) + 5
F32, F8 = torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(wr, "load_library", lambda: lib)
    monkeypatch.setattr(block, "_lib", lambda: lib)
    monkeypatch.setattr(block, "_fast", block._Nothing())
    monkeypatch.setattr(block, "_current", lambda index: 0)
    monkeypatch.setattr(wr, "_stream", lambda dev, stream: None)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Fake(1))
    yield
    assert not lib.calls


CASES = {
    "scan_fwd T": lambda: wr.delta_scan_fwd(Fake(1, BIG, 8), Fake(1, BIG, 8)),
    "scan_fwd B": lambda: wr.delta_scan_fwd(Fake(BIG, 1, 8), Fake(BIG, 1, 8)),
    "scan_step D": lambda: wr.delta_scan_step(Fake(1, BIG), Fake(1, BIG), Fake(1, BIG, dtype=F32)),
    "scan_bwd": lambda: wr.delta_scan_bwd(Fake(1, BIG, 8), Fake(1, BIG, 8), Fake(1, -(-BIG // 64), 8, dtype=F32),
                                          Fake(1, BIG, 8)),
    "norm_fwd D": lambda: wr.delta_add_rmsnorm_fwd(Fake(2, BIG), Fake(BIG)),
    "norm_quant D": lambda: wr.delta_add_rmsnorm_quant(Fake(2, BIG), Fake(BIG)),
    "norm_bwd D": lambda: wr.delta_add_rmsnorm_bwd(Fake(2, BIG), Fake(2, BIG), Fake(BIG), Fake(2, dtype=F32)),
    "linear M": lambda: wr.delta_linear_fwd(Fake(BIG, 8), Fake(16, 8)),
    "linear M of axes": lambda: wr.delta_linear_fwd(Fake(1 << 16, 1 << 16, 8), Fake(16, 8)),
    "linear N": lambda: wr.delta_linear_fwd(Fake(2, 8), Fake(BIG, 8)),
    "linear K": lambda: wr.delta_linear_fwd(Fake(2, BIG), Fake(16, BIG)),
    "linear_quant M": lambda: wr.delta_linear_quant(Fake(BIG, 16, dtype=F8), Fake(BIG, dtype=F32),
                                                    Fake(16, 16, dtype=F8), Fake(16, dtype=F32)),
    "linear_bwd M": lambda: wr.delta_linear_bwd(Fake(BIG, 8), Fake(16, 8), Fake(BIG, 16)),
    "fwd T": lambda: wr.delta_fwd(Fake(1, BIG, 1, 16), Fake(1, BIG, 1, 16), Fake(1, BIG, 1, 16),
                                  Fake(1, BIG, 1, dtype=F32)),
    "fwd dv": lambda: wr.delta_fwd(Fake(1, 2, 1, 16), Fake(1, 2, 1, 16), Fake(1, 2, 1, (1 << 32) + 64),
                                   Fake(1, 2, 1, dtype=F32)),
    "step B": lambda: wr.delta_step(Fake(BIG, 1, 16), Fake(BIG, 1, 1, 16), Fake(BIG, 1, 1, 16),
                                    Fake(BIG, 1, 1, dtype=F32), None, Fake(BIG, 1, 16, 16, dtype=F32)),
    "erank B": lambda: wr.delta_state_erank(Fake(BIG, 1, 16, 16, dtype=F32)),
    "ut T": lambda: wr.delta_ut_transform(Fake(1, BIG, 1, 128), Fake(1, BIG, 1, dtype=F32)),
}


@pytest.mark.parametrize("name", CASES)
def test_refused(name):
    with pytest.raises(ValueError, match="the most is 2\\^31 - 1"):
        CASES[name]()
