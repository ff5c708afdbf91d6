"""The compiled calls of the block operators and the checked Python ones give
the same results, and take the same arguments."""
import pytest
import torch

import weight_rnn_gb300 as wr
from weight_rnn_gb300 import block

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.fixture
def both(monkeypatch):
    """Runs a call through either way and compares the outputs bit by bit."""
    def run(call):
        fast = flat(call())
        monkeypatch.setattr(block, "_fast", block._Nothing())
        slow = flat(call())
        monkeypatch.undo()
        torch.cuda.synchronize()
        assert len(fast) == len(slow)
        for a, b in zip(fast, slow):
            assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride()
            assert torch.equal(a.view(torch.uint8) if a.dtype == block.E4M3 else a,
                               b.view(torch.uint8) if b.dtype == block.E4M3 else b)
    return run


def test_binding_was_built():
    assert not isinstance(block._open_fast(), block._Nothing)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_both_ways_agree(both, dtype):
    r = lambda *s: torch.randn(*s, device="cuda").to(dtype)
    B, T, D = 2, 130, 48
    wide = r(B, T, 2 * D)
    x, g, h0 = wide[..., :D], wide[..., D:], torch.randn(B, D, device="cuda")
    n = torch.tensor([5, 130], device="cuda", dtype=torch.int32)
    lin = torch.rand(B, T, D, device="cuda")
    both(lambda: wr.delta_scan_fwd(x, g, h0, lengths=n, save_states=True))
    both(lambda: wr.delta_scan_fwd(x, lin, form="linear", save_states=1))
    states = wr.delta_scan_fwd(x, g, h0, save_states=True)[2]
    both(lambda: wr.delta_scan_bwd(x, g, states, r(B, T, D) * 0 + 1, h0, lengths=n))
    both(lambda: wr.delta_scan_bwd(x, lin, states, x.contiguous(), form="linear"))
    both(lambda: wr.delta_scan_step(x[:, 0], g[:, 0], h0.clone()))
    w, bw = torch.rand(D, device="cuda"), torch.rand(D, device="cuda").to(BF)
    rows = wide.view(B * T, 2 * D)[:, :D]
    for weight in (w, bw):
        both(lambda: wr.delta_add_rmsnorm_fwd(rows, weight, rows))
        both(lambda: wr.delta_add_rmsnorm_fwd(wide[0, 0, :D], weight))
        both(lambda: wr.delta_add_rmsnorm_quant(x.contiguous(), weight, x.contiguous()))
    _, s, rstd = wr.delta_add_rmsnorm_fwd(x.contiguous(), w, x.contiguous())
    both(lambda: wr.delta_add_rmsnorm_bwd(x.contiguous(), s, w, rstd, s))
    both(lambda: wr.delta_add_rmsnorm_bwd(x.contiguous(), s, w, rstd))
    W, b = r(72, D), torch.rand(72, device="cuda")
    res = r(B, T, 72)
    both(lambda: wr.delta_linear_fwd(x.contiguous(), W, b, res, act="silu", save_pre=True))
    both(lambda: wr.delta_linear_fwd(rows, W, act="gelu"))
    both(lambda: wr.delta_linear_fwd(x[0, 0], W, b.to(BF)))
    both(lambda: wr.delta_linear_bwd(x.contiguous(), W, res, res, act="silu"))
    both(lambda: wr.delta_linear_bwd(rows, W, res.view(B * T, 72), want=(0, 1, False)))
    q, k = x.contiguous().to(block.E4M3), W.to(block.E4M3)
    sx, sw = torch.rand(B, T, device="cuda"), torch.rand(72, device="cuda")
    both(lambda: wr.delta_linear_quant(q, sx, k, sw, b, res.to(BF), act="gelu"))


def test_wrong_arguments_say_what_is_wrong():
    x = torch.zeros(2, 4, 8, device="cuda", dtype=BF)
    w = torch.ones(8, device="cuda")
    lin = torch.zeros(16, 8, device="cuda", dtype=BF)
    cases = [
        (ValueError, "gate has shape", lambda: wr.delta_scan_fwd(x, x[:, :2])),
        (TypeError, "gate has dtype", lambda: wr.delta_scan_fwd(x, x, form="linear")),
        (ValueError, "form must be", lambda: wr.delta_scan_fwd(x, x, form="cubic")),
        (ValueError, "last axis of x", lambda: wr.delta_scan_fwd(x.transpose(1, 2), x.transpose(1, 2))),
        (TypeError, "lengths has dtype", lambda: wr.delta_scan_fwd(
            x, x, lengths=torch.zeros(2, device="cuda", dtype=torch.int64))),
        (TypeError, "x must be bfloat16 or float32", lambda: wr.delta_scan_fwd(x.half(), x.half())),
        (ValueError, "state must be contiguous", lambda: wr.delta_scan_step(
            x[:, 0], x[:, 0], torch.zeros(8, 2, device="cuda").t())),
        (ValueError, "states has shape", lambda: wr.delta_scan_bwd(x, x, w, x)),
        (ValueError, "weight has shape", lambda: wr.delta_add_rmsnorm_fwd(x, w[:4])),
        (wr.DeltaError, "eps", lambda: wr.delta_add_rmsnorm_fwd(x, w, eps=0.0)),
        (wr.DeltaError, "built for D <= 8192", lambda: wr.delta_add_rmsnorm_fwd(
            torch.zeros(1, 8200, device="cuda"), torch.zeros(8200, device="cuda"))),
        (ValueError, "sum_out needs a residual", lambda: wr.delta_add_rmsnorm_fwd(x, w, sum_out=x)),
        (ValueError, "act must be", lambda: wr.delta_linear_fwd(x, lin, act="relu")),
        (ValueError, "x has shape", lambda: wr.delta_linear_fwd(x[..., :4], lin)),
        (ValueError, "residual has shape", lambda: wr.delta_linear_fwd(x, lin, None, x)),
        (TypeError, "pre must be", lambda: wr.delta_linear_bwd(x, lin, torch.zeros(2, 4, 16, device="cuda", dtype=BF),
                                                               act="silu")),
        (TypeError, "x has dtype", lambda: wr.delta_linear_quant(x, w, lin, w)),
        (ValueError, "expected cuda", lambda: wr.delta_linear_fwd(x, lin.cpu())),
    ]
    for kind, text, call in cases:
        with pytest.raises(kind, match=text):
            call()
    wr.delta_inject_failure(1)
    with pytest.raises(wr.DeltaError, match="injected"):
        wr.delta_scan_fwd(x, x)
