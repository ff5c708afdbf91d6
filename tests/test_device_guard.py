"""Tensors on a device that is not the current one: the library is called with
theirs current, and what was current stays so."""
import pytest
import torch

import weight_rnn_gb300 as wr
from fakes import Fake, Library
from weight_rnn_gb300 import block

F32, F8 = torch.float32, torch.float8_e4m3fn


@pytest.fixture
def devices(monkeypatch):
    """Two devices, of which 0 is current; notes where the library was called."""
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
    monkeypatch.setattr(wr, "load_library", lambda: lib)
    monkeypatch.setattr(block, "_lib", lambda: lib)
    monkeypatch.setattr(block, "_fast", block._Nothing())
    monkeypatch.setattr(block, "_current", lambda index: 0)
    monkeypatch.setattr(wr, "_stream", lambda dev, stream: None)
    monkeypatch.setattr(torch, "empty", lambda *a, dtype=BF, device=None: Fake(*(a[0] if len(a) == 1 else a), dtype=dtype, device=device))
    yield seen
    assert now == [0]


BF = torch.bfloat16


def made(device):
    t = lambda *s, dtype=BF: Fake(*s, dtype=dtype, device=device)
    x, g, h = t(2, 5, 8), t(2, 5, 8), t(2, 8, dtype=F32)
    w, q, k = t(16, 8), t(1, 4, 1, 16), t(1, 4, 1, 16)
    b, one = t(1, 4, 1, dtype=F32), t(1, 1, 16)
    return {
        "delta_scan_fwd": lambda: wr.delta_scan_fwd(x, g, h),
        "delta_scan_step": lambda: wr.delta_scan_step(t(2, 8), t(2, 8), h),
        "delta_scan_bwd": lambda: wr.delta_scan_bwd(x, g, t(2, 1, 8, dtype=F32), x),
        "delta_add_rmsnorm_fwd": lambda: wr.delta_add_rmsnorm_fwd(x, t(8), x),
        "delta_add_rmsnorm_quant": lambda: wr.delta_add_rmsnorm_quant(x, t(8), x),
        "delta_add_rmsnorm_bwd": lambda: wr.delta_add_rmsnorm_bwd(x, x, t(8), t(2, 5, dtype=F32)),
        "delta_linear_fwd": lambda: wr.delta_linear_fwd(x, w),
        "delta_linear_quant": lambda: wr.delta_linear_quant(t(2, 8, dtype=F8), t(2, dtype=F32), t(16, 8, dtype=F8),
                                                            t(16, dtype=F32)),
        "delta_linear_bwd": lambda: wr.delta_linear_bwd(x, w, t(2, 5, 16)),
        "delta_fwd": lambda: wr.delta_fwd(q, k, k, b),
        "delta_bwd": lambda: wr.delta_bwd(q, k, k, b, None, None, q),
        "delta_step": lambda: wr.delta_step(one, t(1, 1, 1, 16), t(1, 1, 1, 16), t(1, 1, 1, dtype=F32), None,
                                            t(1, 1, 16, 16, dtype=F32)),
        "delta_state_erank": lambda: wr.delta_state_erank(t(1, 1, 16, 16, dtype=F32)),
        "delta_attention_map": lambda: wr.delta_attention_map(q, k, b),
    }


@pytest.mark.parametrize("name", made("cuda:0"))
@pytest.mark.parametrize("index", [0, 1])
def test_library_sees_the_tensors_device(devices, name, index):
    made(f"cuda:{index}")[name]()
    assert devices == [(name, index)]
