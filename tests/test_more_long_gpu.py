"""Layer norm, the gated layer and decay attention on tensors of more than 2^31 elements:
what is far behind in memory has the values that it has in a tensor of its own."""
import pytest
import torch

import decay_ref
import test_glu_gpu as glu
import test_layernorm_gpu as layernorm
import weight_rnn_gb300 as wr
from block_ref import HALF, U, within
from test_block_long_gpu import TAIL, normal, room  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROWS = 560_000


def test_layernorm():
    D = 4096
    x, r, dy = normal(ROWS, D), normal(ROWS, D), normal(ROWS, D)
    assert x.numel() > 1 << 31
    w, b = torch.rand(D, device="cuda") + 0.5, torch.randn(D, device="cuda")
    got = wr.delta_add_layernorm_fwd(x, w, b, r, eps=layernorm.EPS)
    cpu = lambda t: t[-TAIL:].cpu()  # noqa: E731
    layernorm.check([cpu(t) for t in got], cpu(x), cpu(r), w.cpu(), b.cpu())
    dy[:-TAIL] = 0  # the weights' gradients are the tail's
    back = wr.delta_add_layernorm_bwd(dy, got[1], w, got[2], got[3])
    (dx, dw, db), (big, bigw, bigb) = layernorm.gradients(*(cpu(t) for t in (dy, *got[1:])), w.cpu(), None)
    within(back[0][-TAIL:], dx, 64 * U * big + HALF[BF] * (dx.abs() + 64 * U * big), "dx")
    within(back[1], dw, (TAIL + 48) * U * bigw, "dweight")
    within(back[2], db, (TAIL + 48) * U * bigb, "dbias")
    assert not back[0][:TAIL].any()


def test_glu():
    M, N, K = ROWS, 2048, 64
    x, w, b, _ = glu.inputs(TAIL, N, K, BF, 9)
    big = normal(M, K)
    big[-TAIL:] = x.cuda()
    out, pre = wr.delta_glu_fwd(big, w.cuda(), b.cuda(), save_pre=True)
    assert pre.numel() > 1 << 31
    glu.check(out[-TAIL:], pre[-TAIL:], x, w, b, "silu")
    do = normal(M, N)
    do[:-TAIL] = 0  # so that dw and dbias are the tail's too
    got = wr.delta_glu_bwd(big, w.cuda(), do, pre)
    glu.gradients((got[0][-TAIL:], got[1], None), x, w, do[-TAIL:].cpu(), pre[-TAIL:].cpu(), "silu")
    assert not got[0][:TAIL].any()
    wr.delta_check_device()


def test_decay_in_float32():
    B, T, H, d, n = 1, (1 << 20) + 70, 32, 64, 700
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(B, T, H, d, generator=gen, device="cuda") for _ in range(3))
    assert q.numel() > 1 << 31
    decay = torch.full((H,), 0.5, device="cuda")  # 300 tokens back nothing is left in float32
    out, hT = wr.delta_decay_fwd(q, k, v, decay)
    ro, rh, bo, bh = decay_ref.forward(*(t[:, -n:, -2:].cpu() for t in (q, k, v)), decay[:2].cpu())
    within(out[:, -300:, -2:], ro[:, -300:], decay_ref.out_error(ro, bo, T, d, torch.float32, False)[:, -300:], "out")
    within(hT[:, -2:], rh, bh * decay_ref.slack(T, 1, False), "hT")
