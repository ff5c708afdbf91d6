"""Rows without elements: what there is one of a row is still given a value."""
import pytest
import torch

import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_rows_of_no_elements(residual, side):
    torch.full((1 << 20,), float("nan"), device="cuda")  # freed: what an allocation may hold
    stream = torch.cuda.Stream() if side else None
    x, w = torch.zeros(70, 5, 0, device="cuda"), torch.zeros(0, device="cuda")
    r = x.clone() if residual else None
    y, total, rstd = wr.delta_add_rmsnorm_fwd(x, w, r, eps=0.25, stream=stream)
    q, scale, _ = wr.delta_add_rmsnorm_quant(x, w, r, stream=stream)
    torch.cuda.synchronize()
    assert y.shape == total.shape == q.shape == (70, 5, 0)
    assert torch.equal(rstd, torch.full((70, 5), 2.0, device="cuda"))
    assert torch.equal(scale, torch.ones(70, 5, device="cuda"))
    dx, dw = wr.delta_add_rmsnorm_bwd(y, total, w, rstd)
    assert dx.shape == (70, 5, 0) and dw.shape == (0,)
