"""Layer norm of rows whose squares, or whose plain sum, pass float32's range: they count
as infinitely wide, rstd 0 and y = bias, with the mean that they have; their gradient is
dsum, and they add nothing to the weight's."""
import pytest
import torch

import weight_rnn_gb300 as wr
from block_ref import U, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def rows_of(D, dtype):
    """finite elements, whose plain sums are not"""
    i = torch.arange(D)
    most = 3.3e38
    x = torch.stack([
        torch.where(i % 2 == 0, 1e35, 2e35) * (8192 / D),   # one sign
        torch.where(i % 2 == 0, -3e38, -1e38),
        torch.where(i % 3 == 0, most, 0.5 * most),
        torch.where(i % 2 == 0, most, -most),               # a mean near 0
        torch.where(i == D // 2, -most, most),              # a difference past the range
        torch.where(i < D // 2, most, -0.9 * most),         # warps whose own means are far apart
    ])
    return x.to(dtype)


# several rows to a warp, one, several warps a row; pairs and single elements
@pytest.mark.parametrize("D", [8, 64, 128, 512, 1024, 4096, 8192, 50, 2050, 1001, 8191])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_past_the_range(D, dtype, residual):
    gen = torch.Generator().manual_seed(D)
    x = rows_of(D, dtype)
    x = torch.cat([x, torch.randn(3, D, generator=gen).to(dtype)])  # and rows like others beside them
    n = len(x) - 3
    w, b = 1.0 + torch.rand(D, generator=gen), torch.randn(D, generator=gen)
    r = torch.zeros_like(x) if residual else None
    y, total, mean, rstd = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), r if r is None else r.cuda(), eps=EPS)
    assert torch.equal(total.cpu(), x)
    t = x.double()
    # chains of at most 40 roundings of the mean magnitude, and the quotient
    within(mean, t.mean(-1), 41 * U * t.abs().mean(-1) + 1e-38, "mean")
    assert not rstd[:n].any()
    assert torch.equal(y[:n].cpu(), b.to(dtype).expand(n, D))
    dy, ds = (torch.randn(len(x), D, generator=gen).to(dtype) for _ in range(2))
    dx, dw, db = wr.delta_add_layernorm_bwd(dy.cuda(), total, w.cuda(), mean, rstd, ds.cuda())
    assert torch.equal(dx[:n].cpu(), ds[:n])
    that = (t[n:] - mean[n:].cpu().double()[:, None]) * rstd[n:].cpu().double()[:, None]
    terms = dy[n:].double() * that
    within(dw, terms.sum(0), (len(x) + 48) * U * terms.abs().sum(0) + 1e-38, "dweight")
    within(db, dy.double().sum(0), (len(x) + 48) * U * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_infinite_rows_stay_not_numbers(dtype):
    """An element that is infinite is no wide row: the norm has no value."""
    x = torch.ones(4, 512, dtype=dtype)
    x[1, 7], x[2, 9] = float("inf"), -float("inf")
    y, _, _, rstd = wr.delta_add_layernorm_fwd(x.cuda(), torch.ones(512, device="cuda"))
    assert torch.isnan(y[1:3]).all() and torch.isnan(rstd[1:3]).all()
    assert not y[0].any() and not y[3].any()


@pytest.mark.parametrize("D", [1, 2, 3, 8, 64, 65, 1000, 1024, 1025, 8192])
def test_tiny_rows_keep_their_mean(D):
    """Elements near the end of float32's normal range, and below it: sums are of elements
    over D's power of two, and lose at most 2^-150 in each of 40 roundings, which is less
    than 2^-143 of the mean."""
    x = torch.randn(6, D, generator=torch.Generator().manual_seed(D)).abs() + 1.0
    x *= torch.tensor([1e-30, 1e-34, 1e-36, 1e-37, 1.2e-38, 1e-40])[:, None]
    y, _, mean, _ = wr.delta_add_layernorm_fwd(x.cuda(), torch.ones(D, device="cuda"), eps=EPS)
    t = x.double()
    within(mean, t.mean(-1), 41 * U * t.abs().mean(-1) + 2.0 ** -143, "mean")
    assert (y.abs().cpu() <= 1e-25).all()
