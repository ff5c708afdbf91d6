"""The block operators on tensors of more than 2^31 elements: what is far behind
in memory has the values that it has in a tensor of its own."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr
from test_linear_gpu import check, gradients
from test_norm_gpu import EPS, K as KN, check as check_norm

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ROWS, TAIL = 560_000, 64


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 120e9:
        pytest.skip("needs 120 GB")
    yield
    torch.cuda.empty_cache()


def normal(*shape):
    return torch.empty(*shape, dtype=BF, device="cuda").normal_()


def test_scan():
    B, T, D, n = 2, 1_100_032, 2048, 2048
    x, gate = normal(B, T, D), normal(B, T, D)
    out, hT, states = wr.delta_scan_fwd(x, gate, save_states=True)
    # sigmoid gates of normal logits forget: 1024 steps multiply by less than e^-400
    to, th, ts = wr.delta_scan_fwd(x[1:, -n:], gate[1:, -n:], save_states=True)
    far, near = out[1, -n // 2:].double(), to[0, -n // 2:].double()
    # two sums in other orders, within 1e-5 of each other, each rounded by half a step
    assert ((far - near).abs() <= 2.0 ** -7 * near.abs() + 1e-5).all()
    assert ((hT[1] - th[0]).abs() <= 1e-5).all()
    dx, dg, _ = wr.delta_scan_bwd(x, gate, states, out)
    tx, tg, _ = wr.delta_scan_bwd(x[1:, -n:], gate[1:, -n:], states[1:, -n // 64:].contiguous(),
                                  out[1:, -n:].contiguous())
    for a, b in ((dx, tx), (dg, tg)):
        far, near = a[1, -n:].double(), b[0].double()
        assert ((far - near).abs() <= 2.0 ** -7 * near.abs() + 1e-4).all()
    wr.delta_check_device()


def test_norm():
    D = 4096
    x, r, w = normal(ROWS, D), normal(ROWS, D), torch.rand(D, device="cuda") + 0.5
    got = wr.delta_add_rmsnorm_fwd(x, w, r, eps=EPS)
    q, scale, _ = wr.delta_add_rmsnorm_quant(x, w, r, eps=EPS)
    xt, rt, wt = x[-TAIL:].cpu(), r[-TAIL:].cpu(), w.cpu()
    check_norm([t[-TAIL:] for t in got], xt, rt, wt)
    y = ref.norm(xt, rt, wt, EPS)[2]
    step = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * scale[-TAIL:].cpu().double()[:, None])
    ref.within(q[-TAIL:].float().double() * scale[-TAIL:].double()[:, None], y, step * (1 + 4 * KN) + 4 * KN * y.abs(),
               "8 bits")
    x[:-TAIL] = 0  # as dy: the weight's gradient is the tail's
    dx, dw = wr.delta_add_rmsnorm_bwd(x, got[1], w, got[2])
    (want, wantw), (big, bigw) = ref.norm_grad(xt, got[1][-TAIL:].cpu(), wt, got[2][-TAIL:].cpu(), None)
    ref.within(dx[-TAIL:], want, KN * big + ref.HALF[BF] * (want.abs() + KN * big), "dx")
    ref.within(dw, wantw, (TAIL + 48) * ref.U * bigw, "dweight")
    assert not dx[:-TAIL].any()
    wr.delta_check_device()


def test_linear_outputs_and_gradients():
    N, K = 4096, 64
    x, w = normal(ROWS, K), normal(N, K) / 8
    b = torch.randn(N, device="cuda")
    out, pre = wr.delta_linear_fwd(x, w, b, act="silu", save_pre=True)
    torch.cuda.synchronize()
    wr.delta_check_device()
    for rows in (slice(0, TAIL), slice(ROWS - TAIL, ROWS)):
        check(out[rows].cpu(), pre[rows].cpu(), x[rows].cpu(), w.cpu(), b.cpu(), None, "silu")
    out[:-TAIL] = 0  # as dout
    dx, dw, db = wr.delta_linear_bwd(x, w, out, pre, act="silu")
    torch.cuda.synchronize()
    wr.delta_check_device()
    assert not dx[:-TAIL].any()
    gradients((dx[-TAIL:].cpu(), dw, db), x[-TAIL:].cpu(), w.cpu(), out[-TAIL:].cpu(), pre[-TAIL:].cpu(), "silu")


@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_linear_inputs(dtype):
    N, K = 72, 4096
    x, w = normal(ROWS, K).to(dtype), (normal(N, K) / 64).to(dtype)
    if dtype == BF:
        out, scales = wr.delta_linear_fwd(x, w), None
    else:
        sx, sw = torch.rand(ROWS, device="cuda") + 0.1, torch.rand(N, device="cuda") + 0.1
        out, scales = wr.delta_linear_quant(x, sx, w, sw), (sx[-TAIL:].cpu(), sw.cpu())
    torch.cuda.synchronize()
    wr.delta_check_device()
    check(out[-TAIL:].cpu(), None, x[-TAIL:].cpu().float(), w.cpu().float(), None, None, "none", scales)
