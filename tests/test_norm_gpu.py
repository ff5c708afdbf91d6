"""GPU parity of the residual addition with RMS norm (delta_add_rmsnorm_*) with
its 64-bit definition.  Float32 adds at most: the sum's rounding, about 40 for
the mean of squares (chains of up to 16 elements a thread, 5 shuffles and 16
warps, halved by the root), 4 for the root and 2 products; 64 roundings U are
allowed in all.  An output's own rounding is half a step."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
K = 64 * ref.U
EPS = 1e-5
within = ref.within

SHAPES = [(1, 1), (3, 7), (1, 4096), (2, 8192), (5, 8191), (700, 64), (700, 72), (513, 1001),
          (4, 2050), (1300, 2048), (400, 4100), (1, 256), (37, 520)]


def inputs(rows, D, dtype, seed, wdtype=F32):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x, res = r(rows, D).to(dtype), (3.0 * r(rows, D)).to(dtype)
    return x, res, (1.0 + 0.3 * r(D)).to(wdtype), r(rows, D).to(dtype), r(rows, D).to(dtype)


def check(got, x, res, w):
    t, rstd, y = ref.norm(x, res, w, EPS)
    half = ref.HALF[x.dtype]
    within(got[0], y, (K + half * (1 + K)) * y.abs() + 1e-38, "y")
    within(got[1], t, (ref.U + half) * t.abs(), "sum")
    within(got[2], rstd, K * rstd, "rstd")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    x, res, w, _, _ = inputs(*shape, dtype, sum(shape), BF if shape[0] % 2 else F32)
    got = wr.delta_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    plain = wr.delta_add_rmsnorm_fwd(x.cuda(), w.cuda(), eps=EPS)
    torch.cuda.synchronize()
    check(got, x, res, w)
    check(plain, x, None, w)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_eight_bits(shape, dtype):
    x, res, w, _, _ = inputs(*shape, dtype, sum(shape) + 1)
    if shape[0] > 2:
        x[1], res[1] = 0, 0  # a row of zeros
    q, scale, total = wr.delta_add_rmsnorm_quant(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    torch.cuda.synchronize()
    t, _, y = ref.norm(x, res, w, EPS)
    want = y.abs().amax(-1) / 448.0
    want = torch.where(want > 0, want, torch.ones_like(want))
    within(scale, want, 2 * K * want, "scale")
    within(total, t, (ref.U + ref.HALF[dtype]) * t.abs(), "sum")
    value = q.cpu().double() * scale.cpu().double()[:, None]
    # e4m3: half a step is 2^-4 of the value, or 2^-10 below its normal range
    step = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * want[:, None])
    within(value, y, step * (1 + 4 * K) + 4 * K * y.abs(), "value")
    if shape[0] > 2:
        assert scale[1].item() == 1.0 and not q[1].float().any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, dtype):
    x, res, w, dy, ds = inputs(*shape, dtype, sum(shape) + 2)
    _, total, rstd = wr.delta_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    both = wr.delta_add_rmsnorm_bwd(dy.cuda(), total, w.cuda(), rstd, ds.cuda())
    alone = wr.delta_add_rmsnorm_bwd(dy.cuda(), total, w.cuda(), rstd)
    again = wr.delta_add_rmsnorm_bwd(dy.cuda(), total, w.cuda(), rstd, ds.cuda())
    torch.cuda.synchronize()
    for got, d in ((both, ds), (alone, None)):
        (dx, dw), (big, bigw) = ref.norm_grad(dy, total.cpu(), w, rstd.cpu(), d)
        within(got[0], dx, K * big + ref.HALF[dtype] * (dx.abs() + K * big), "dx")
        within(got[1], dw, (shape[0] + 48) * ref.U * bigw, "dweight")
    assert torch.equal(both[0], again[0]) and torch.equal(both[1], again[1])


def test_in_place_and_strided_rows():
    x, res, w, dy, ds = inputs(90, 128, BF, 5)
    for shift in (0, 8, 3):  # aligned vectors, and single elements
        wide = torch.zeros(90, 300, device="cuda", dtype=BF)
        xv = wide[:, shift:shift + 128]
        xv.copy_(x)
        stream = res.cuda()
        got = wr.delta_add_rmsnorm_fwd(xv, w.cuda(), stream, eps=EPS, sum_out=stream)
        torch.cuda.synchronize()
        assert got[1] is stream
        check(got, x, res, w)
        g, d = dy.cuda(), ds.cuda()
        want = wr.delta_add_rmsnorm_bwd(g, stream, w.cuda(), got[2], d)
        a = wr.delta_add_rmsnorm_bwd(g.clone(), stream, w.cuda(), got[2], d, dx=d)
        assert a[0] is d and torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])


def test_three_axes_and_no_rows():
    x, res, w, dy, _ = inputs(12, 40, F32, 6)
    shape = (3, 4, 40)
    got = wr.delta_add_rmsnorm_fwd(x.cuda().view(shape), w.cuda(), res.cuda().view(shape), eps=EPS)
    torch.cuda.synchronize()
    assert got[0].shape == shape and got[2].shape == (3, 4)
    check([t.reshape(12, *t.shape[2:]) for t in got], x, res, w)
    part = torch.zeros(4, 5, 40, device="cuda")[:, :2]
    with pytest.raises(ValueError, match="fold"):
        wr.delta_add_rmsnorm_fwd(part, w.cuda())
    none = torch.zeros(0, 40, device="cuda")
    y, _, rstd = wr.delta_add_rmsnorm_fwd(none, w.cuda())
    assert y.shape == (0, 40) and rstd.shape == (0,)
    dx, dw = wr.delta_add_rmsnorm_bwd(none, none, w.cuda(), rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros_like(dw))


def test_nan_and_infinity_stay_in_their_row():
    x, res, w, dy, _ = inputs(400, 64, BF, 7)
    x[3, 5], x[9, 1] = float("nan"), float("inf")
    got = wr.delta_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    q, _, _ = wr.delta_add_rmsnorm_quant(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    torch.cuda.synchronize()
    keep = [i for i in range(400) if i not in (3, 9)]
    check([t.cpu()[keep] for t in got], x[keep], res[keep], w)
    assert torch.isnan(got[0][3]).all() and torch.isnan(got[0][9, 1])
    assert torch.isnan(q[3].float()).all() and torch.isfinite(q.float()[keep]).all()


def test_graph_and_side_stream():
    x, res, w, dy, ds = inputs(600, 1024, BF, 8)
    gx, gr, gw, gd, gs = (t.cuda() for t in (x, res, w, dy, ds))
    want = wr.delta_add_rmsnorm_fwd(gx, gw, gr)
    wgrad = wr.delta_add_rmsnorm_bwd(gd, want[1], gw, want[2], gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    grad = wr.delta_add_rmsnorm_bwd(gd, want[1], gw, want[2], gs, stream=side)
    side.synchronize()
    assert torch.equal(grad[0], wgrad[0]) and torch.equal(grad[1], wgrad[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wr.delta_add_rmsnorm_fwd(gx, gw, gr)
        grads = wr.delta_add_rmsnorm_bwd(gd, out[1], gw, out[2], gs)
    for t in (*out, *grads):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((*out, *grads), (*want, *wgrad)):
        assert torch.equal(p, q)
