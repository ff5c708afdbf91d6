"""GPU parity of the linear layer (delta_linear_*) with its 64-bit definition.

Bounds per element.  A tensor-core product adds 16 (bfloat16) or 32 (e4m3)
terms at a time to a float32 sum, truncating at worst: a step (2 U) of the sum
of magnitudes for each, plus a few for the parts that meet (split k).  The
epilogue adds a handful of roundings and the hardware exponential (2^-22 and
its argument's rounding); the activations' slopes are below 1.13.  In the
gradients dpre is rounded to the operands' type, half a step of each term."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = ref.U
within = ref.within


def chain(K):
    return 2 * U * (K / 16 + 24)


def rel(got, want):
    d = (got.cpu().double() - want).norm()
    n = want.norm()
    return (d / n).item() if n > 0 else d.item()


def inputs(M, N, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return (r(M, K).to(dtype), (r(N, K) / K ** 0.5).to(dtype), 0.5 * r(N), r(M, N).to(dtype),
            r(M, N).to(dtype))


def pad(t, extra, fill=float("nan")):
    """the same matrix as a slice of wider rows, on the GPU"""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=torch.float32).to(t.dtype).cuda()
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def check(out, pre, x, w, b, res, act, scales=None):
    xd, wd = x.double(), w.double()
    if scales is not None:
        xd, wd = xd * scales[0].double()[:, None], wd * scales[1].double()[:, None]
    p, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    bias = 0.0 if b is None else b.double()
    ep = chain(x.shape[1]) * mag + 8 * U * (mag + (0.0 if b is None else b.double().abs()))
    p = p + bias
    half = ref.HALF[out.dtype]
    if pre is not None:
        within(pre, p, ep + half * (p.abs() + ep), "pre")
    o = ref.act(act, p)
    eo = 1.13 * ep + (2.0 ** -20 * (1.0 + p.abs()) * p.abs() if act != "none" else 0.0)
    if res is not None:
        o = o + res.double()
        eo = eo + U * o.abs()
    within(out, o, eo + half * (o.abs() + eo), "out")


# gradients on both sides of the bound of the one-launch form, sums over 1..8 CTAs
MIDDLE = [(1, 512, 512), (64, 512, 512), (100, 101, 102), (513, 40, 64), (260, 515, 333), (2816, 19, 257), (40, 1100, 330)]
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (3, 17, 7), (8, 128, 200), (9, 100, 1024), (16, 257, 72),
          (17, 513, 130), (31, 40, 513), (32, 2048, 512), (33, 64, 64), (64, 65, 8), (100, 257, 63),
          (127, 8, 1000), (129, 300, 65), (300, 520, 1000), (257, 1024, 2048),
          (40, 131, 700), (520, 72, 1500), (200, 900, 4096), (90, 2000, 530),
          # past the small products: odd rows to pack, odd widths to store, k split with both
          (700, 333, 401), (260, 1003, 300), (3000, 257, 129), (128, 4096, 257), (40, 1999, 1001)]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_bf16(shape, act):
    x, w, b, res, _ = inputs(*shape, BF, sum(shape))
    bias = b if shape[0] % 2 else b.to(BF)
    out, pre = wr.delta_linear_fwd(x.cuda(), w.cuda(), bias.cuda(), res.cuda(), act=act, save_pre=True)
    bare = wr.delta_linear_fwd(x.cuda(), w.cuda(), act=act)
    torch.cuda.synchronize()
    wr.delta_check_device()
    check(out, pre, x, w, bias, res, act)
    check(bare, None, x, w, None, None, act)


@pytest.mark.parametrize("shape", [(1300, 5000, 72), (2500, 1300, 136), (5000, 264, 40)], ids=str)
def test_many_tiles_a_cta(shape):
    x, w, b, res, _ = inputs(*shape, BF, 3)
    out, pre = wr.delta_linear_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), act="silu", save_pre=True)
    again = wr.delta_linear_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), act="silu")
    torch.cuda.synchronize()
    wr.delta_check_device()
    check(out, pre, x, w, b, res, "silu")
    assert torch.equal(out, again)


@pytest.mark.parametrize("shape", SHAPES + [(2500, 1300, 136), (2100, 2600, 264)], ids=str)
def test_eight_bits(shape):
    M, N, K = shape
    x, w, b, res, _ = inputs(*shape, F32, sum(shape) + 7)
    sx, sw = x.abs().amax(1) / 448, w.abs().amax(1) / 448
    q, k = (x / sx[:, None]).to(E4M3), (w / sw[:, None]).to(E4M3)
    res = res.to(BF)
    out = wr.delta_linear_quant(q.cuda(), sx.cuda(), k.cuda(), sw.cuda(), b.cuda(), res.cuda(), act="gelu")
    bare = wr.delta_linear_quant(q.cuda(), sx.cuda(), k.cuda(), sw.cuda())
    torch.cuda.synchronize()
    wr.delta_check_device()
    check(out, None, q.float(), k.float(), b, res, "gelu", (sx, sw))
    check(bare, None, q.float(), k.float(), None, None, "none", (sx, sw))


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 70, 33), (65, 64, 130), (130, 200, 17)], ids=str)
def test_forward_and_gradients_f32(shape):
    M, N, K = shape
    x, w, b, res, do = inputs(*shape, F32, sum(shape))
    out, pre = wr.delta_linear_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), act="silu", save_pre=True)
    got = wr.delta_linear_bwd(x.cuda(), w.cuda(), do.cuda(), pre, act="silu")
    torch.cuda.synchronize()
    xd, wd = x.double(), w.double()
    p, mag = xd @ wd.T + b.double(), xd.abs() @ wd.abs().T + b.double().abs()
    ep = U * (K + 8) * mag
    within(pre, p, ep, "pre")
    o = ref.act("silu", p) + res.double()
    within(out, o, 1.13 * ep + 2.0 ** -20 * (1 + p.abs()) * p.abs() + 2 * U * o.abs(), "out")
    gradients(got, x, w, do, pre.cpu(), "silu")


def gradients(got, x, w, do, pre, act):
    p = (torch.zeros_like(do) if pre is None else pre).double().requires_grad_(True)
    dpre = do.double() if act == "none" else torch.autograd.grad(ref.act(act, p), p, do.double())[0]
    xd, wd = x.double(), w.double()
    # the slope's own error: its terms are below 1 + |p|, each good to about
    # 2^-20 of (1 + |p|); then dpre's rounding to the operands' type
    es = 0.0 if act == "none" else 2.0 ** -19 * do.double().abs() * (1 + p.detach().abs()) ** 2
    half = ref.HALF[x.dtype]
    e = es + (0.0 if act == "none" else half * (dpre.abs() + es))
    n = (lambda k: chain(k)) if x.dtype == BF else (lambda k: U * (k + 8))
    for name, g, want, mag, err, k in (
            ("dx", got[0], dpre @ wd, dpre.abs() @ wd.abs(), None if act == "none" else e @ wd.abs(), w.shape[0]),
            ("dw", got[1], dpre.T @ xd, dpre.abs().T @ xd.abs(), None if act == "none" else e.T @ xd.abs(),
             x.shape[0])):
        if g is None:
            continue
        bound = n(k) * mag + (0.0 if err is None else 1.01 * err)
        within(g, want, bound + half * (want.abs() + bound) + 1e-38, name)
        # of the whole: two roundings, each within half a step
        assert rel(g, want) <= 2 * half + 1e-5, name
    if got[2] is not None:
        es_sum = es.sum(0) if act != "none" else 0.0
        within(got[2], dpre.sum(0), U * (x.shape[0] + 40) * dpre.abs().sum(0) + es_sum + 1e-38, "dbias")


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] < 1000] + [(300, 2600, 2100), (2100, 300, 2600)] + MIDDLE, ids=str)
def test_gradients_bf16(shape, act):
    x, w, b, _, do = inputs(*shape, BF, sum(shape) + 1)
    pre = None if act == "none" else (x.float() @ w.float().T + b).to(BF)
    args = (x.cuda(), w.cuda(), do.cuda(), None if pre is None else pre.cuda())
    got = wr.delta_linear_bwd(*args, act=act)
    again = wr.delta_linear_bwd(*args, act=act)
    part = wr.delta_linear_bwd(*args, act=act, want=(False, True, False))
    rest = wr.delta_linear_bwd(*args, act=act, want=(True, False, False))
    sums = wr.delta_linear_bwd(*args, act=act, want=(False, False, True))
    torch.cuda.synchronize()
    wr.delta_check_device()
    gradients(got, x, w, do, pre, act)
    for a, c in zip(got, again):
        assert torch.equal(a, c)
    assert part[0] is None and part[2] is None and torch.equal(part[1], got[1])
    assert torch.equal(rest[0], got[0]) and torch.equal(sums[2], got[2])


@pytest.mark.parametrize("M,N", [(5, 72), (150, 72), (1500, 520)])
@pytest.mark.parametrize("extra", [1, 8, 24])
def test_strided_rows_read_nothing_beside_them(M, N, extra):
    K = 136
    x, w, b, res, do = inputs(M, N, K, BF, 21)
    xp, wp, rp = pad(x, extra), pad(w, extra), pad(res, extra)
    out, pre = wr.delta_linear_fwd(xp, wp, b.cuda(), rp, act="silu", save_pre=True)
    got = wr.delta_linear_bwd(xp, wp, do.cuda(), pre, act="silu")
    torch.cuda.synchronize()
    check(out, pre, x, w, b, res, "silu")
    gradients(got, x, w, do, pre.cpu(), "silu")
    sx, sw = torch.rand(M) + 0.1, torch.rand(N) + 0.1
    q, k = x.to(E4M3), w.to(E4M3)
    out = wr.delta_linear_quant(pad(q, extra), sx.cuda(), pad(k, extra), sw.cuda(), act="silu")
    torch.cuda.synchronize()
    check(out, None, q.float(), k.float(), None, None, "silu", (sx, sw))


@pytest.mark.parametrize("M", [4, 200, 6000])
def test_in_place_residual_and_leading_axes(M):
    x, w, b, res, _ = inputs(2 * M, 64, 128, BF, 5)
    stream = res.cuda().view(2, M, 64)
    out = wr.delta_linear_fwd(x.cuda().view(2, M, 128), w.cuda(), b.cuda(), stream, act="gelu", out=stream)
    torch.cuda.synchronize()
    assert out is stream
    check(out.view(2 * M, 64), None, x, w, b, res, "gelu")


def test_nan_and_infinity_stay_in_their_rows():
    for M in (8, 160, 6000):
        x, w, b, res, _ = inputs(M, 96, 160, BF, 6)
        x[2, 3], x[5, 100] = float("nan"), float("inf")
        out = wr.delta_linear_fwd(x.cuda(), w.cuda(), b.cuda(), res.cuda(), act="silu")
        torch.cuda.synchronize()
        keep = [i for i in range(M) if i not in (2, 5)]
        check(out.cpu()[keep], None, x[keep], w, b, res[keep], "silu")
        assert torch.isnan(out[2]).all() and not torch.isfinite(out[5]).all()


def test_empty_sizes():
    w, x = torch.zeros(8, 16, device="cuda", dtype=BF), torch.zeros(0, 16, device="cuda", dtype=BF)
    assert wr.delta_linear_fwd(x, w).shape == (0, 8)
    dx, dw, db = wr.delta_linear_bwd(x, w, torch.zeros(0, 8, device="cuda", dtype=BF))
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def test_gradient_against_differences_of_the_kernel():
    # without an activation the layer is linear in each argument: a difference
    # over any span is the derivative, up to the outputs' roundings
    x, w, b, _, do = inputs(200, 96, 128, BF, 9)
    g = [t.cuda() for t in (x, w, do)]
    dx, dw, db = wr.delta_linear_bwd(g[0], g[1], g[2])
    v, u = torch.randn(200, 128, device="cuda").to(BF), torch.randn(96, 128, device="cuda").to(BF)
    loss = lambda x, w: (wr.delta_linear_fwd(x, w).double() * g[2]).sum()
    for num, ana in ((loss(v, g[1]), (dx.double() * v).sum()), (loss(g[0], u), (dw.double() * u).sum())):
        # 19200 roundings of at most 2^-8 of terms of size ~ sqrt(128): independent, so about
        # sqrt(19200) 2^-8 11 / sqrt(3) = 3.4 on either side; ten of those
        assert abs(num - ana) <= 35.0


@pytest.mark.parametrize("M,N", [(300, 200), (3000, 400)])
def test_graph_and_side_stream(M, N):
    x, w, b, res, do = (t.cuda() for t in inputs(M, N, 72, BF, 10))
    want = wr.delta_linear_fwd(x, w, b, res, act="silu", save_pre=True)
    wgrad = wr.delta_linear_bwd(x, w, do, want[1], act="silu")
    small = wr.delta_linear_fwd(x[:2], w, b, res[:2], act="silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wr.delta_linear_bwd(x, w, do, want[1], act="silu", stream=side)
    side.synchronize()
    for p, q in zip(got, wgrad):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wr.delta_linear_fwd(x, w, b, res, act="silu", save_pre=True)
        grads = wr.delta_linear_bwd(x, w, do, out[1], act="silu")
        tiny = wr.delta_linear_fwd(x[:2], w, b, res[:2], act="silu")
    for t in (*out, *grads, tiny):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((*out, *grads, tiny), (*want, *wgrad, small)):
        assert torch.equal(p, q)
    wr.delta_check_device()
