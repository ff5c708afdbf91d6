"""Decays that are not numbers, or negative, reach every result of their head on all
ways through the forward and the gradients, and nothing else."""
import pytest
import torch

import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# whole rows; a cut time axis; heads that CTAs share; value channels in two groups
@pytest.mark.parametrize("B,T,H,d,dv", [(2, 300, 3, 32, 32), (1, 1500, 2, 64, 64), (5, 300, 40, 32, 32), (1, 130, 2, 16, 136)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), -0.5])
@pytest.mark.parametrize("ragged", [False, True], ids=["whole", "ragged"])
def test_decays_without_a_logarithm(B, T, H, d, dv, dtype, bad, ragged):
    gen = torch.Generator(device="cuda").manual_seed(B)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = (normal(B, T, H, n).to(dtype) for n in (d, d, dv, dv))
    h0, dh = normal(B, H, d, dv), normal(B, H, d, dv)
    decay = 0.5 + 0.5 * torch.rand(H, generator=gen, device="cuda")
    broken = decay.clone()
    broken[1] = bad
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    if ragged:
        n[0], n[-1] = T - 150 if T > 150 else 1, 0
        if B == 1:
            n[0] = T - 129
    lengths = n if ragged else None
    call = lambda g: (*wr.delta_decay_fwd(q, k, v, g, h0, lengths=lengths),  # noqa: E731
                      *wr.delta_decay_bwd(q, k, v, g, do, h0, dh, lengths=lengths))
    want, got = call(decay), call(broken)
    wr.delta_check_device()
    others = [h for h in range(H) if h != 1]
    live = torch.arange(T, device="cuda") < n[:, None]
    for name, a, b in zip(("out", "hT", "dq", "dk", "dv", "dh0"), got, want):
        state = name in ("hT", "dh0")
        axis = 1 if state else 2
        assert torch.equal(a.select(axis, 0), b.select(axis, 0)), name
        idx = torch.tensor(others, device="cuda")
        assert torch.equal(a.index_select(axis, idx), b.index_select(axis, idx)), name
        head, was = a.select(axis, 1), b.select(axis, 1)
        counts = n > 0 if state else live
        sure = counts
        if name in ("dk", "dv"):  # (nothing is decayed on its way to a row's last token)
            sure = live & (torch.arange(T, device="cuda") < n[:, None] - 1)
        assert torch.isnan(head[sure]).all(), name
        assert torch.equal(head[~counts], was[~counts]), name  # no token: the state as it was, out 0


def test_step_takes_the_decay_as_it_is():
    gen = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, state = normal(2, 3, 16), normal(2, 3, 16), normal(2, 3, 8), normal(2, 3, 16, 8)
    decay = torch.tensor([float("nan"), -0.5, 1.0], device="cuda")
    want = decay[:, None, None] * state + k[..., None] * v[..., None, :]
    out = wr.delta_decay_step(q, k, v, decay, state)
    assert torch.isnan(out[:, 0]).all() and torch.isnan(state[:, 0]).all()
    torch.testing.assert_close(state[:, 1:], want[:, 1:], rtol=1e-6, atol=1e-6)
    torch.testing.assert_close(out[:, 1:], (q[..., None] * want).sum(-2)[:, 1:], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,d", [(300, 32), (1500, 64)])
def test_what_dout_holds_past_a_row_does_not_matter(T, d, dtype, bad):
    gen = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    n = torch.tensor([0, 1, 129, T - 1], dtype=torch.int32, device="cuda")
    q, k, v, do = (normal(4, T, 2, d).to(dtype) for _ in range(4))
    decay, h0, dh = torch.tensor([0.9, 1.0], device="cuda"), normal(4, 2, d, d), normal(4, 2, d, d)
    want = wr.delta_decay_bwd(q, k, v, decay, do, h0, dh, lengths=n)
    past = torch.arange(T, device="cuda") >= n[:, None]
    spoiled = [t.masked_fill(past[:, :, None, None], bad) for t in (q, k, v, do)]
    got = wr.delta_decay_bwd(*spoiled[:3], decay, spoiled[3], h0, dh, lengths=n)
    wr.delta_check_device()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
