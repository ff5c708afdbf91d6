"""The 64-bit definitions that the block operators' GPU tests compare with,
pinned on the CPU: closed forms and finite differences."""
import pytest
import torch

import block_ref as ref


def _scan_inputs(form, seed=0, B=2, T=9, D=3):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    gate = r(B, T, D) if form == "sigmoid" else torch.rand(B, T, D, generator=gen, dtype=torch.float64)
    return r(B, T, D), gate, r(B, D), r(B, T, D), r(B, D)


@pytest.mark.parametrize("form", ["linear", "sigmoid"])
def test_scan_closed_form(form):
    x, gate, h0, _, _ = _scan_inputs(form)
    a, u = (gate, torch.ones_like(gate)) if form == "linear" else (gate.sigmoid(), 1 - gate.sigmoid())
    out, hT, _, _, _ = ref.scan(x, gate, h0, None, form)
    T = x.shape[1]
    want = a.prod(1) * h0 + sum(a[:, s + 1:].prod(1) * (u * x)[:, s] for s in range(T))
    torch.testing.assert_close(hT, want, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(out[:, -1], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("form", ["linear", "sigmoid"])
@pytest.mark.parametrize("lengths", [None, [9, 0], [4, 20]])
def test_scan_gradient_is_the_difference_quotient(form, lengths):
    x, gate, h0, dout, dhT = _scan_inputs(form, 1)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)

    def loss(x, gate, h0):
        out, hT, _, _, _ = ref.scan(x, gate, h0, n, form)
        return (out * dout).sum() + (hT * dhT).sum()

    grads, _ = ref.scan_grad(x, gate, h0, dout, dhT, n, form)
    gen = torch.Generator().manual_seed(2)
    for i, g in enumerate(grads):
        args = [x, gate, h0]
        v = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        e = 1e-6
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + e * v, args[i] - e * v
        num = (loss(*hi) - loss(*lo)) / (2 * e)
        assert abs(num - (g * v).sum()) <= 1e-7 * (1 + abs(num))


def test_reset_drops_nan_and_inf():
    x = torch.ones(1, 4, 2, dtype=torch.float64)
    x[0, 0, 0], x[0, 1, 1] = float("nan"), float("inf")
    gate = torch.full_like(x, 0.5)
    gate[0, 2] = 0.0
    out, hT, _, _, _ = ref.scan(x, gate, None, None, "linear")
    assert torch.equal(out[0, 2], torch.ones(2, dtype=torch.float64))
    assert torch.equal(hT[0], torch.full((2,), 1.5, dtype=torch.float64))


def test_norm_gradient_is_the_difference_quotient():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, res, w, dy, ds = r(3, 7), r(3, 7), r(7), r(3, 7), r(3, 7)
    eps = 1e-3
    t, rstd, _ = ref.norm(x, res, w, eps)
    (dx, dw), _ = ref.norm_grad(dy, t, w, rstd, ds)

    def loss(x, w):
        t, _, y = ref.norm(x, res, w, eps)
        return (y * dy).sum() + (t * ds).sum()

    for g, args, i in ((dx, (x, w), 0), (dw, (x, w), 1)):
        v = r(*args[i].shape)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-6 * v, args[i] - 1e-6 * v
        num = (loss(*hi) - loss(*lo)) / 2e-6
        assert abs(num - (g * v).sum()) <= 1e-7 * (1 + abs(num))
