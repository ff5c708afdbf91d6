"""The activations' derivatives over the whole range of what a layer keeps before
them, in the kernels that form them: one launch for small layers, the pass
before the tensor-core products, and float32."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MAGNITUDES = [0.0, 0.125, 0.75, 1.5, 3.0, 5.0, 8.0, 12.0, 16.0, 17.0, 40.0, 100.0, 1e4, 1e10, 1.9e19, 1e20, 1e30, 3e38]


def bound(act, p):
    """The logistic function is good to 2^-21 (two hardware operations), 1 - s to
    2^-24 on top, each of six further operations to 2^-24."""
    c, k = (8.0 / torch.pi) ** 0.5, 0.044715
    if act == "none":
        return torch.zeros_like(p)
    s = torch.special.expit(p if act == "silu" else c * (p + k * p ** 3))
    # an argument's own rounding, 2^-22 of it, moves s by s (1 - s) times that
    arg = p.abs() if act == "silu" else c * (p.abs() + k * p.abs() ** 3)
    ds = s * 2.0 ** -21 + s * (1 - s) * arg * 2.0 ** -22
    near = p.abs().clamp(max=100.0)
    rise = near if act == "silu" else near * c * (1 + 3 * k * near ** 2)
    live = (s * (1 - s) > 2.0 ** -60).double()  # elsewhere the second term is 0 in float32 too
    return ds + live * rise * (2 * ds + s * 2.0 ** -23) + s * (1 - s) * rise * 6 * 2.0 ** -24 + 2.0 ** -60


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype,M,N,K", [(BF, 1, 36, 64), (BF, 3, 36, 64), (BF, 700, 2088, 2048), (F32, 3, 36, 40)])
def test_slope_of_any_size(act, dtype, M, N, K):
    pre = torch.tensor([v for m in MAGNITUDES for v in (m, -m)]).repeat(-(-N // 36))[:N].to(dtype).expand(M, N).contiguous()
    gen = torch.Generator().manual_seed(N)
    x, w = (torch.randn(*s, generator=gen).to(dtype) for s in ((M, K), (N, K)))
    dout = torch.zeros(M, N, dtype=dtype)
    dout[M // 2] = 1.0  # one row's slopes are the bias's gradient
    dx, dw, db = wr.delta_linear_bwd(x.cuda(), w.cuda(), dout.cuda(), pre.cuda(), act=act)
    torch.cuda.synchronize()
    p = pre[0].double().requires_grad_(True)
    (slope,) = torch.autograd.grad(ref.act(act, p).sum(), p)
    p = p.detach()
    ref.within(db, slope, bound(act, p), "dbias")
    # dpre may be rounded once to the operands' type, and the outputs are
    half, dp = ref.HALF[dtype], bound(act, p)
    wd, xd = w.double(), x[M // 2].double()
    want = slope @ wd
    big = (slope.abs() @ wd.abs())
    ref.within(dx[M // 2], want, dp @ wd.abs() + big * (half + (N + 8) * ref.U) + half * want.abs(), "dx")
    want = slope[:, None] * xd
    ref.within(dw, want, (dp[:, None] + slope.abs()[:, None] * (half + (M + 8) * ref.U)) * xd.abs() * (1 + half)
               + half * want.abs(), "dw")
