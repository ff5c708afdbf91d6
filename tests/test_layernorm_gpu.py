"""GPU parity of the residual addition with layer norm (delta_add_layernorm_*) with its
64-bit definition.  What float32 adds, in roundings U: the sum's own one; the mean, a
sum in chains of at most 16 elements a thread, 5 shuffles and 16 warps, 40 of the mean
magnitude m1; the differences, one more, and the mean's error in each; the variance, 40
for its sum, and twice the mean's error over the deviation, whose square is all that
stays of it where the deviations add up to 0, so that rstd is off by 64 U and by
(40 U m1 / s)^2, s the deviation.  The sum's rounding, U |t| an element, moves the
variance by 2 mean(c e) for differences c and roundings e, which is at most 2 U rms(c)
rms(t), and rstd by half of that times rstd^2.  An output's own rounding is half a
step."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = ref.U
EPS = 1e-5
within = ref.within

SHAPES = [(1, 1), (3, 7), (1, 4096), (2, 8192), (5, 8191), (700, 64), (700, 72), (513, 1001),
          (4, 2050), (1300, 2048), (400, 4100), (1, 256), (37, 520),
          # several rows to a warp
          (1000, 128), (1001, 16), (65, 32), (7, 8), (5000, 40), (333, 120), (1, 64), (1363, 2)]


def inputs(rows, D, dtype, seed, wdtype=F32):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, res = r(rows, D).to(dtype), (3.0 * r(rows, D) + r(rows, 1)).to(dtype)
    w, b = (1.0 + 0.3 * r(D)).to(wdtype), r(D).to(BF if wdtype == F32 else F32)
    return x, res, w, b, r(rows, D).to(dtype), r(rows, D).to(dtype)


def stats(t):
    m1 = t.abs().mean(-1)
    mean = t.mean(-1)
    var = (t - mean[..., None]).square().mean(-1)
    rstd = (var + EPS).rsqrt()
    moved = U * (var * t.square().mean(-1)).sqrt() * rstd ** 2
    return mean, rstd, 41 * U * m1, 64 * U + 4 * (41 * U * m1 * rstd) ** 2 + moved


def check(got, x, res, w, b):
    t = x.double() + (0.0 if res is None else res.double())
    mean, rstd, em, er = stats(t)
    half = ref.HALF[x.dtype]
    c = t - mean[:, None]
    b = torch.zeros_like(w) if b is None else b
    y = c * rstd[:, None] * w.double() + b.double()
    lost = ((er[:, None] + 4 * U) * c.abs() + em[:, None] + 2 * U * t.abs()) * rstd[:, None] * w.double().abs()
    lost = lost * (1 + 100 * U) + 2 * U * y.abs()
    within(got[0], y, lost + half * (y.abs() + lost) + 1e-38, "y")
    within(got[1], t, (U + half) * t.abs(), "sum")
    within(got[2], mean, em + 1e-38, "mean")
    within(got[3], rstd, er * rstd, "rstd")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    x, res, w, b, _, _ = inputs(*shape, dtype, sum(shape), BF if shape[0] % 2 else F32)
    got = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), eps=EPS)
    plain = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), eps=EPS)
    torch.cuda.synchronize()
    check(got, x, res, w, b)
    check(plain, x, None, w, None)


def test_a_mean_far_from_zero():
    """Deviations of 1 on a mean of 4096: mean t^2 - mean^2 would lose 24 bits here."""
    x, _, w, b, _, _ = inputs(300, 2048, F32, 3)
    x = x + 4096.0
    got = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    check(got, x, None, w, b)


def gradients(dy, total, mean, rstd, w, ds):
    """dx, dweight, dbias and the magnitudes of their terms"""
    m, r = mean.double()[:, None], rstd.double()[:, None]
    c, g = total.double() - m, dy.double() * w.double()
    that = c * r
    d = torch.zeros_like(g) if ds is None else ds.double()
    mu = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    dx = r * (g - mu(g) - that * mu(g * that)) + d
    big = r * (g.abs() + mu(g.abs()) + that.abs() * mu((g * that).abs())) + d.abs()
    return (dx, (dy.double() * that).sum(0), dy.double().sum(0)), \
        (big, (dy.double() * that).abs().sum(0), dy.double().abs().sum(0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, dtype):
    x, res, w, b, dy, ds = inputs(*shape, dtype, sum(shape) + 2)
    _, total, mean, rstd = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), eps=EPS)
    both = wr.delta_add_layernorm_bwd(dy.cuda(), total, w.cuda(), mean, rstd, ds.cuda())
    alone = wr.delta_add_layernorm_bwd(dy.cuda(), total, w.cuda(), mean, rstd)
    again = wr.delta_add_layernorm_bwd(dy.cuda(), total, w.cuda(), mean, rstd, ds.cuda())
    torch.cuda.synchronize()
    for got, d in ((both, ds), (alone, None)):
        (dx, dw, db), (big, bigw, bigb) = gradients(dy, total.cpu(), mean.cpu(), rstd.cpu(), w, d)
        within(got[0], dx, 64 * U * big + ref.HALF[dtype] * (dx.abs() + 64 * U * big) + 1e-38, "dx")
        within(got[1], dw, (shape[0] + 48) * U * bigw, "dweight")
        within(got[2], db, (shape[0] + 48) * U * bigb, "dbias")
    assert all(torch.equal(p, q) for p, q in zip(both, again))


def test_gradients_are_the_forwards_slopes():
    """Central differences of y . dy + sum . ds in the 64-bit definition."""
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, dy, ds = r(6, 40).float(), r(40).float(), r(40).float(), r(6, 40).float(), r(6, 40).float()
    _, total, mean, rstd = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    got = wr.delta_add_layernorm_bwd(dy.cuda(), total, w.cuda(), mean, rstd, ds.cuda())

    def loss(x, w, b):
        m, s, _, _ = stats(x)
        return (((x - m[:, None]) * s[:, None] * w + b) * dy.double()).sum() + (x * ds.double()).sum()
    args = [t.double() for t in (x, w, b)]
    for i, g in enumerate(got):
        d = r(*args[i].shape)
        step = lambda h: loss(*(a + h * d if j == i else a for j, a in enumerate(args)))  # noqa: E731
        slope = (step(1e-4) - step(-1e-4)) / 2e-4
        want = (g.cpu().double() * d).sum()
        assert abs(slope - want) <= 1e-5 * (g.cpu().double() * d).abs().sum(), i


def test_in_place_and_strided_rows():
    x, res, w, b, dy, ds = inputs(90, 128, BF, 5)
    for shift in (0, 8, 3):  # aligned vectors, and single elements
        wide = torch.zeros(90, 300, device="cuda", dtype=BF)
        xv = wide[:, shift:shift + 128]
        xv.copy_(x)
        stream = res.cuda()
        got = wr.delta_add_layernorm_fwd(xv, w.cuda(), b.cuda(), stream, eps=EPS, sum_out=stream)
        torch.cuda.synchronize()
        assert got[1] is stream
        check(got, x, res, w, b)
        g, d = dy.cuda(), ds.cuda()
        want = wr.delta_add_layernorm_bwd(g, stream, w.cuda(), *got[2:], d)
        a = wr.delta_add_layernorm_bwd(g.clone(), stream, w.cuda(), *got[2:], d, dx=d)
        assert a[0] is d and all(torch.equal(p, q) for p, q in zip(a, want))


def test_three_axes_and_no_rows_and_no_elements():
    x, res, w, b, dy, _ = inputs(12, 40, F32, 6)
    shape = (3, 4, 40)
    got = wr.delta_add_layernorm_fwd(x.cuda().view(shape), w.cuda(), b.cuda(), res.cuda().view(shape), eps=EPS)
    torch.cuda.synchronize()
    assert got[0].shape == shape and got[2].shape == got[3].shape == (3, 4)
    check([t.reshape(12, *t.shape[2:]) for t in got], x, res, w, b)
    none = torch.zeros(0, 40, device="cuda")
    y, _, mean, rstd = wr.delta_add_layernorm_fwd(none, w.cuda(), b.cuda())
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    dx, dw, db = wr.delta_add_layernorm_bwd(none, none, w.cuda(), mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 40) and not dw.any() and not db.any()
    empty = torch.zeros(3, 0, device="cuda")
    _, _, mean, rstd = wr.delta_add_layernorm_fwd(empty, torch.zeros(0, device="cuda"), eps=0.25)
    assert torch.equal(mean, torch.zeros_like(mean)) and torch.equal(rstd, torch.full_like(rstd, 2.0))


def test_constant_rows():
    """No deviation: y is the bias, rstd eps^-1/2."""
    x = torch.full((5, 512), 3.0, dtype=BF)
    w, b = torch.ones(512), torch.arange(512.0)
    y, _, mean, rstd = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    assert torch.equal(y.cpu(), b.to(BF).expand(5, 512)) and torch.equal(mean.cpu(), torch.full((5,), 3.0))
    within(rstd, torch.full((5,), EPS ** -0.5, dtype=torch.float64), 64 * U * EPS ** -0.5 * torch.ones(5), "rstd")


def test_nan_and_infinity_stay_in_their_row():
    x, res, w, b, _, _ = inputs(400, 64, BF, 7)
    x[3, 5], x[9, 1] = float("nan"), float("inf")
    got = wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), eps=EPS)
    torch.cuda.synchronize()
    keep = [i for i in range(400) if i not in (3, 9)]
    check([t.cpu()[keep] for t in got], x[keep], res[keep], w, b)
    assert torch.isnan(got[0][3]).all() and torch.isnan(got[0][9]).all()


def test_graph_and_side_stream():
    x, res, w, b, dy, ds = inputs(600, 1024, BF, 8)
    gx, gr, gw, gb, gd, gs = (t.cuda() for t in (x, res, w, b, dy, ds))
    want = wr.delta_add_layernorm_fwd(gx, gw, gb, gr)
    wgrad = wr.delta_add_layernorm_bwd(gd, want[1], gw, want[2], want[3], gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    grad = wr.delta_add_layernorm_bwd(gd, want[1], gw, want[2], want[3], gs, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(grad, wgrad))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wr.delta_add_layernorm_fwd(gx, gw, gb, gr)
        grads = wr.delta_add_layernorm_bwd(gd, out[1], gw, out[2], out[3], gs)
    for t in (*out, *grads):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((*out, *grads), (*want, *wgrad)):
        assert torch.equal(p, q)


def test_sizes_of_elements():
    """Squares within float32's range up to its end; past it a row counts as infinitely
    wide: rstd is 0 and y the bias."""
    x, _, w, b, _, _ = inputs(6, 512, F32, 11)
    for i, size in enumerate((1e-30, 1e-10, 1e10, 1e17, 1e22, 1e30)):
        x[i] *= size
    got = [t.cpu() for t in wr.delta_add_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)]
    check([t[:4] for t in got], x[:4], None, w, b)
    assert not got[3][4:].any()
    assert torch.equal(got[0][4:], b.float().expand(2, -1))
