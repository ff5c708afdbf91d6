"""GPU parity of the gated layer (delta_glu_*) with its 64-bit definition.

Bounds per element, as for the linear layer: a tensor-core product adds 16 terms at a
time to a float32 sum, truncating at worst, a step (2 U) of the sum of magnitudes for
each and a few for the parts that meet.  act(g) u then has act's error times |u| and
u's times |act(g)|, act's slope being below 1.13, and two more roundings.  In the
gradients dpre is rounded to the operands' type, half a step of each term."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr
from test_slopes_gpu import MAGNITUDES, bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = ref.U
within = ref.within


def chain(K, dtype):
    return 2 * U * (K / 16 + 24) if dtype == BF else U * (K + 8)


def inputs(M, N, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return r(M, K).to(dtype), (r(2 * N, K) / K ** 0.5).to(dtype), 0.5 * r(2 * N), r(M, N).to(dtype)


def pad(t, extra):
    """the same matrix as a slice of wider rows, NaN beside it, on the GPU"""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def check(out, pre, x, w, b, act):
    N = w.shape[0] // 2
    xd, wd = x.double(), w.double()
    p, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    if b is not None:
        p, mag = p + b.double(), mag + b.double().abs()
    ep = (chain(x.shape[1], x.dtype) + 8 * U) * mag
    half = ref.HALF[x.dtype]
    if pre is not None:
        within(pre, p, ep + half * (p.abs() + ep), "pre")
    g, u, eg, eu = p[:, :N], p[:, N:], ep[:, :N], ep[:, N:]
    a = ref.act(act, g)
    ea = 1.13 * eg + (2.0 ** -20 * (1.0 + g.abs()) * g.abs() if act != "none" else 0.0)
    o = a * u
    eo = ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * o.abs()
    within(out, o, eo + half * (o.abs() + eo) + 1e-38, "out")


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (3, 17, 7), (8, 128, 200), (9, 100, 1024), (16, 257, 72),
          (17, 513, 130), (31, 40, 513), (32, 1024, 512), (33, 64, 64), (64, 65, 8), (100, 129, 63),
          (127, 8, 1000), (129, 300, 65), (300, 520, 1000), (257, 1024, 2048), (40, 66, 700), (520, 36, 1500),
          (200, 450, 4096), (90, 1000, 530),
          # past the small products: odd rows to pack, odd widths to store, k split with both
          (700, 333, 401), (260, 503, 300), (3000, 129, 129), (128, 2048, 257), (40, 999, 1001), (128, 96, 4096)]
TILES = [(1300, 2500, 72), (2500, 650, 136), (5000, 132, 40), (4100, 2056, 264), (3000, 1001, 64)]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES + TILES, ids=str)
def test_forward_bf16(shape, act):
    x, w, b, _ = inputs(*shape, BF, sum(shape))
    bias = b if shape[0] % 2 else b.to(BF)
    out, pre = wr.delta_glu_fwd(x.cuda(), w.cuda(), bias.cuda(), act=act, save_pre=True)
    again = wr.delta_glu_fwd(x.cuda(), w.cuda(), bias.cuda(), act=act)
    bare = wr.delta_glu_fwd(x.cuda(), w.cuda(), act=act)
    torch.cuda.synchronize()
    wr.delta_check_device()
    check(out, pre, x, w, bias, act)
    check(bare, None, x, w, None, act)
    assert torch.equal(out, again)


def gradients(got, x, w, do, pre, act):
    N = w.shape[0] // 2
    p = pre.double().requires_grad_(True)
    (dpre,) = torch.autograd.grad(ref.act(act, p[:, :N]) * p[:, N:], p, do.double())
    p, d = p.detach(), do.double().abs()
    # the slope's own error, as for the linear layer, times |u|; act's, about 2^-20 (1 + |g|) |g|
    one = 1.0 + p[:, :N].abs()
    es = torch.cat([2.0 ** -19 * d * p[:, N:].abs() * one ** 2, 2.0 ** -19 * d * one ** 2], 1) + 4 * U * dpre.abs()
    half = ref.HALF[x.dtype]
    e = es + half * (dpre.abs() + es)
    xd, wd = x.double(), w.double()
    for name, g, want, mag, err, k in (
            ("dx", got[0], dpre @ wd, dpre.abs() @ wd.abs(), e @ wd.abs(), w.shape[0]),
            ("dw", got[1], dpre.T @ xd, dpre.abs().T @ xd.abs(), e.T @ xd.abs(), x.shape[0])):
        if g is None:
            continue
        bound = chain(k, x.dtype) * mag + 1.01 * err
        within(g, want, bound + half * (want.abs() + bound) + 1e-38, name)
        # of the whole: two roundings, each within half a step
        assert (g.cpu().double() - want).norm() <= (2 * half + 1e-5) * want.norm() + 1e-38, name
    if got[2] is not None:
        within(got[2], dpre.sum(0), U * (x.shape[0] + 40) * dpre.abs().sum(0) + es.sum(0) + 1e-38, "dbias")


MIDDLE = [(1, 256, 512), (64, 256, 512), (100, 51, 102), (513, 20, 64), (260, 257, 333), (2816, 10, 257), (40, 550, 330),
          (300, 1300, 2100), (2100, 150, 2600)]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] < 1000] + MIDDLE, ids=str)
def test_gradients_bf16(shape, act):
    x, w, b, do = inputs(*shape, BF, sum(shape) + 1)
    pre = (x.float() @ w.float().T + b).to(BF)
    args = (x.cuda(), w.cuda(), do.cuda(), pre.cuda())
    got = wr.delta_glu_bwd(*args, act=act)
    again = wr.delta_glu_bwd(*args, act=act)
    part = wr.delta_glu_bwd(*args, act=act, want=(False, True, False))
    rest = wr.delta_glu_bwd(*args, act=act, want=(True, False, False))
    sums = wr.delta_glu_bwd(*args, act=act, want=(False, False, True))
    torch.cuda.synchronize()
    wr.delta_check_device()
    gradients(got, x, w, do, pre, act)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    assert part[0] is None and part[2] is None and torch.equal(part[1], got[1])
    assert torch.equal(rest[0], got[0]) and torch.equal(sums[2], got[2])


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 35, 33), (65, 32, 130), (130, 100, 17), (70, 129, 65)], ids=str)
def test_forward_and_gradients_f32(shape, act):
    x, w, b, do = inputs(*shape, F32, sum(shape))
    out, pre = wr.delta_glu_fwd(x.cuda(), w.cuda(), b.cuda(), act=act, save_pre=True)
    bare = wr.delta_glu_fwd(x.cuda(), w.cuda(), b.cuda(), act=act)
    got = wr.delta_glu_bwd(x.cuda(), w.cuda(), do.cuda(), pre, act=act)
    torch.cuda.synchronize()
    check(out, pre, x, w, b, act)
    assert torch.equal(out, bare)
    gradients(got, x, w, do, pre.cpu(), act)


@pytest.mark.parametrize("M,N", [(5, 72), (150, 72), (1500, 520)])
@pytest.mark.parametrize("extra", [1, 8, 24])
def test_strided_rows_read_nothing_beside_them(M, N, extra):
    x, w, b, do = inputs(M, N, 136, BF, 21)
    xp, wp = pad(x, extra), pad(w, extra)
    out, pre = wr.delta_glu_fwd(xp, wp, b.cuda(), save_pre=True)
    got = wr.delta_glu_bwd(xp, wp, do.cuda(), pre)
    torch.cuda.synchronize()
    check(out, pre, x, w, b, "silu")
    gradients(got, x, w, do, pre.cpu(), "silu")


@pytest.mark.parametrize("M", [8, 160, 6000])
def test_nan_and_infinity_stay_in_their_rows_and_columns(M):
    x, w, b, _ = inputs(M, 96, 160, BF, 6)
    x[2, 3], w[96 + 7, 5] = float("nan"), float("inf")  # a row of x; a row of the second half
    out = wr.delta_glu_fwd(x.cuda(), w.cuda(), b.cuda())
    torch.cuda.synchronize()
    keep, cols = [i for i in range(M) if i != 2], [j for j in range(96) if j != 7]
    check(out.cpu()[keep][:, cols], None, x[keep], w[cols + [96 + j for j in cols]], b[cols + [96 + j for j in cols]], "silu")
    assert torch.isnan(out[2]).all() and not torch.isfinite(out[:, 7]).any()


@pytest.mark.parametrize("M", [4, 200, 6000])
def test_leading_axes_and_given_output(M):
    x, w, b, _ = inputs(2 * M, 64, 128, BF, 5)
    out = torch.empty(2, M, 64, dtype=BF, device="cuda")
    got = wr.delta_glu_fwd(x.cuda().view(2, M, 128), w.cuda(), b.cuda(), act="gelu", out=out)
    torch.cuda.synchronize()
    assert got is out
    check(out.view(2 * M, 64), None, x, w, b, "gelu")


def test_empty_sizes():
    w, x = torch.zeros(8, 16, device="cuda", dtype=BF), torch.zeros(0, 16, device="cuda", dtype=BF)
    out, pre = wr.delta_glu_fwd(x, w, save_pre=True)
    assert out.shape == (0, 4) and pre.shape == (0, 8)
    dx, dw, db = wr.delta_glu_bwd(x, w, out, pre)
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    none = torch.zeros(0, 16, device="cuda", dtype=BF)
    assert wr.delta_glu_fwd(torch.zeros(3, 16, device="cuda", dtype=BF), none).shape == (3, 0)


@pytest.mark.parametrize("M,N", [(300, 200), (3000, 400)])
def test_graph_and_side_stream(M, N):
    x, w, b, do = (t.cuda() for t in inputs(M, N, 72, BF, 10))
    want = wr.delta_glu_fwd(x, w, b, save_pre=True)
    wgrad = wr.delta_glu_bwd(x, w, do, want[1])
    small = wr.delta_glu_fwd(x[:2], w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wr.delta_glu_bwd(x, w, do, want[1], stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, wgrad))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wr.delta_glu_fwd(x, w, b, save_pre=True)
        grads = wr.delta_glu_bwd(x, w, do, out[1])
        tiny = wr.delta_glu_fwd(x[:2], w, b)
    for t in (*out, *grads, tiny):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((*out, *grads, tiny), (*want, *wgrad, small)):
        assert torch.equal(p, q)
    wr.delta_check_device()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype,M,N,K", [(BF, 3, 72, 64), (BF, 300, 72, 64), (BF, 1500, 2088, 512), (F32, 5, 72, 40)])
def test_ends_of_the_activations_range(act, dtype, M, N, K):
    """Gates of every size, through weights that each copy one element of a row; the other
    half is 1.5.  The value's error is |g| times the logistic function's (test_slopes_gpu),
    which is 0 where it is below float32's range."""
    g = torch.tensor([v for m in MAGNITUDES for v in (m, -m)]).repeat(-(-N // 36))[:N].to(dtype)
    x, w = torch.zeros(M, K, dtype=dtype), torch.zeros(2 * N, K, dtype=dtype)
    x[:, 0], w[:N, 0], w[N:, 0] = 1.0, g, 1.5
    out, pre = wr.delta_glu_fwd(x.cuda(), w.cuda(), act=act, save_pre=True)
    dout = torch.zeros(M, N, dtype=dtype)
    dout[M // 2] = 1.0
    dx, dw, db = wr.delta_glu_bwd(x.cuda(), w.cuda(), dout.cuda(), pre, act=act)
    p = g.double().requires_grad_(True)
    value = ref.act(act, p)
    (slope,) = torch.autograd.grad(value.sum(), p)
    p, value = p.detach(), value.detach()
    c, k = (8.0 / torch.pi) ** 0.5, 0.044715
    s = torch.special.expit(p if act == "silu" else c * (p + k * p ** 3))
    arg = p.abs() if act == "silu" else c * (p.abs() + k * p.abs() ** 3)
    ev = p.abs() * (s * 2.0 ** -21 + s * (1 - s) * arg * 2.0 ** -22 + 2.0 ** -125) + U * value.abs()
    es, half = bound(act, p), ref.HALF[dtype]
    within(pre, torch.cat([p, torch.full_like(p, 1.5)]).expand(M, 2 * N), 0.0, "pre")
    eo = 1.5 * ev + U * (1.5 * value).abs()
    o = torch.where(1.5 * value > torch.finfo(dtype).max, torch.inf, 1.5 * value)  # 1.5 times 3e38 has no value
    within(out, o.expand(M, N), eo + half * (1.5 * value.abs() + eo), "out")
    d = torch.cat([1.5 * slope, value])
    e = torch.cat([1.5 * es, ev]) + 2 * U * d.abs()
    within(db, d, e, "dbias")
    want = d[:, None] * x[M // 2].double()
    e = (e + half * (d.abs() + e))[:, None] * x[M // 2].double()  # dpre is rounded, and dw
    within(dw, want, e + half * (want.abs() + e), "dw")


@pytest.mark.parametrize("glu", [True, False])
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 2048), (2600, 3000, 5000), (5000, 1300, 4104), (3001, 4100, 2570), (9000, 2048, 1500)])
def test_gradients_together_are_those_alone(M, N, K, glu):
    """Large layers have both products in one launch where that is shorter: the same sums,
    also of some rows and columns in 64 bits."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x, do = r(M, K), r(M, N)
    w, pre = (r(2 * N, K), r(M, 2 * N)) if glu else (r(N, K), r(M, N))
    fn = wr.delta_glu_bwd if glu else wr.delta_linear_bwd
    got = fn(x, w, do, pre, act="silu")
    dx = fn(x, w, do, pre, act="silu", want=(True, False, False))[0]
    dw = fn(x, w, do, pre, act="silu", want=(False, True, False))[1]
    wr.delta_check_device()
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    p = pre.double().requires_grad_(True)
    out = ref.act("silu", p[:, :N]) * p[:, N:] if glu else ref.act("silu", p)
    (dpre,) = torch.autograd.grad(out, p, do.double())
    rows, cols = [0, 127, 128, 255, M // 2, M - 1], [0, 129, w.shape[0] // 2, w.shape[0] - 1]
    # two roundings, each within half a step, of the whole of what is looked at
    for name, g, want in (("dx", dx[rows], dpre[rows] @ w.double()), ("dw", dw[cols], dpre[:, cols].T @ x.double())):
        assert (g.double() - want).norm() <= (2 * ref.HALF[BF] + 1e-5) * want.norm(), name
