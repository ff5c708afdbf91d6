"""GPU parity of the gated linear recurrence (delta_scan_*) with its 64-bit
definition.  Bounds are derived per element: block_ref.roundings counts what
float32 adds along the recurrence, and an output's own rounding is half a step."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, D, dtype, form, seed, h0=True, resets=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = r(B, T, D).to(dtype)
    if form == "sigmoid":
        gate = (r(B, T, D) * 2.0 + 2.0).to(dtype)
        if resets and T > 2:  # a logit of -inf is a gate of exactly 0, one of +inf exactly 1
            gate[:, T // 2] = float("-inf")
            gate[:, T // 3] = float("inf")
    else:
        gate = 1.0 - 0.2 * torch.rand(B, T, D, generator=gen) * torch.rand(B, 1, D, generator=gen)
        if resets and T > 2:
            gate[:, T // 2] = 0.0
            gate[:, 1] = -0.7
    return x, gate, (r(B, D) if h0 else None), r(B, T, D).to(dtype), r(B, D)


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_fwd(got, x, gate, h0, lengths, form, states=True):
    out, hT, before, err, _ = ref.scan(x, gate, h0, lengths, form)
    within(got[0], out, err + ref.HALF[x.dtype] * (out.abs() + err), "out")
    last = err[:, -1] if err.shape[1] else 0.0 * hT
    within(got[1], hT, last, "hT")
    if states:
        eb = torch.cat([torch.zeros_like(err[:, :1]), err[:, :-1]], 1)
        within(got[2], before[:, ::64], eb[:, ::64], "states")


within = ref.within

# odd lengths around the tile (64), the warp's 8 steps and a cluster's tiles;
# odd widths around the 32- and 64-channel strips
SHAPES = [(1, 1, 1), (2, 7, 3), (3, 8, 64), (2, 63, 33), (1, 64, 128), (2, 65, 66), (1, 129, 31),
          (2, 511, 40), (1, 1000, 97), (5, 70, 258), (1, 2049, 64)]


@pytest.mark.parametrize("form", ["sigmoid", "linear"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradients(shape, dtype, form):
    x, gate, h0, dout, dhT = inputs(*shape, dtype, form, seed=sum(shape), resets=True)
    dx_, dg_, dh_, do_, dt_ = dev(x, gate, h0, dout, dhT)
    got = wr.delta_scan_fwd(dx_, dg_, dh_, form=form, save_states=True)
    grads = wr.delta_scan_bwd(dx_, dg_, got[2], do_, dt_, form=form)
    torch.cuda.synchronize()
    check_fwd(got, x, gate, h0, None, form)
    want, err = ref.scan_grad(x, gate, h0, dout, dhT, None, form)
    for name, g, w, e, half in zip(("dx", "dgate", "dh0"), grads, want, err,
                                   (ref.HALF[dtype], ref.HALF[gate.dtype], ref.U)):
        within(g, w, e + half * (w.abs() + e) + 1e-40, name)


# enough rows and strips that one CTA walks each alone, and few enough that
# clusters of every size split the time axis
@pytest.mark.parametrize("B,T,D", [(40, 200, 520), (12, 300, 512), (5, 300, 512), (3, 600, 510), (1, 700, 70), (1, 4500, 70)])
@pytest.mark.parametrize("dtype,form", [(BF, "sigmoid"), (F32, "linear")])
def test_every_split_of_time_agrees(B, T, D, dtype, form):
    x, gate, h0, dout, dhT = inputs(B, T, D, dtype, form, seed=T)
    gx, gg, gh, gd, gt = dev(x, gate, h0, dout, dhT)
    got = wr.delta_scan_fwd(gx, gg, gh, form=form, save_states=True)
    grads = wr.delta_scan_bwd(gx, gg, got[2], gd, gt, form=form)
    again = wr.delta_scan_fwd(gx, gg, gh, form=form, save_states=True)
    gagain = wr.delta_scan_bwd(gx, gg, got[2], gd, gt, form=form)
    torch.cuda.synchronize()
    for p, q in zip((*got, *grads), (*again, *gagain)):
        assert torch.equal(p, q)  # the same bits every time
    rows = [0, B - 1]
    sub = lambda t: t[rows]
    check_fwd([sub(g.cpu()) for g in got], sub(x), sub(gate), sub(h0), None, form)
    want, err = ref.scan_grad(sub(x), sub(gate), sub(h0), sub(dout), sub(dhT), None, form)
    for name, g, w, e, half in zip(("dx", "dgate", "dh0"), grads, want, err,
                                   (ref.HALF[dtype], ref.HALF[gate.dtype], ref.U)):
        within(sub(g.cpu()), w, e + half * (w.abs() + e) + 1e-40, name)


@pytest.mark.parametrize("form", ["sigmoid", "linear"])
@pytest.mark.parametrize("T,D", [(130, 64), (77, 35)])
def test_ragged_rows_read_nothing_past_their_length(T, D, form):
    lengths = torch.tensor([0, 1, 64, T - 1, T, T + 100, -3], dtype=torch.int32)
    x, gate, h0, dout, dhT = inputs(len(lengths), T, D, BF, form, seed=9)
    clean = [t.clone() for t in (x, gate, dout)]
    for b, n in enumerate(lengths.clamp(0, T).tolist()):
        for t in (x, gate, dout):
            t[b, n:] = float("nan")
        for t in clean:
            t[b, n:] = 0
    gx, gg, gh, gd, gt, gl = dev(x, gate, h0, dout, dhT, lengths)
    got = wr.delta_scan_fwd(gx, gg, gh, form=form, lengths=gl, save_states=True)
    grads = wr.delta_scan_bwd(gx, gg, got[2], gd, gt, form=form, lengths=gl)
    torch.cuda.synchronize()
    check_fwd(got, clean[0], clean[1], h0, lengths, form)
    want, err = ref.scan_grad(clean[0], clean[1], h0, clean[2], dhT, lengths, form)
    for name, g, w, e, half in zip(("dx", "dgate", "dh0"), grads, want, err,
                                   (ref.HALF[BF], ref.HALF[gate.dtype], ref.U)):
        within(g, w, e + half * (w.abs() + e) + 1e-40, name)


@pytest.mark.parametrize("form", ["sigmoid", "linear"])
def test_slices_of_a_wider_projection(form):
    B, T, D = 2, 90, 64
    x, gate, h0, dout, dhT = inputs(B, T, D, BF, form, seed=4)
    for shift in (0, 1, 2):  # even and odd channel offsets: pairs or single channels
        wide = torch.randn(B, T + 3, 2 * D + 5, device="cuda").to(BF)
        gwide = torch.randn(B, T, 2 * D + 5, device="cuda").to(gate.dtype)
        xv, gv = wide[:, 2:T + 2, shift:shift + D], gwide[:, :, D + shift:2 * D + shift]
        xv.copy_(x)
        gv.copy_(gate)
        got = wr.delta_scan_fwd(xv, gv, h0.cuda(), form=form, save_states=True)
        grads = wr.delta_scan_bwd(xv, gv, got[2], dout.cuda(), dhT.cuda(), form=form)
        torch.cuda.synchronize()
        check_fwd(got, x, gate, h0, None, form)
        want, err = ref.scan_grad(x, gate, h0, dout, dhT, None, form)
        for name, g, w, e, half in zip(("dx", "dgate", "dh0"), grads, want, err,
                                       (ref.HALF[BF], ref.HALF[gate.dtype], ref.U)):
            within(g, w, e + half * (w.abs() + e) + 1e-40, name)


def test_broadcast_batch():
    x, gate, h0, _, _ = inputs(1, 70, 64, F32, "linear", seed=5)
    gx = x.cuda().expand(3, 70, 64)
    out, hT = wr.delta_scan_fwd(gx, gate.cuda().expand(3, 70, 64), None, form="linear")
    torch.cuda.synchronize()
    check_fwd((out, hT), x.expand(3, 70, 64), gate.expand(3, 70, 64), None, None, "linear", states=False)


def test_no_steps_and_in_place_state():
    h0 = torch.randn(3, 40, device="cuda")
    empty = torch.zeros(3, 0, 40, device="cuda", dtype=BF)
    out, hT, states = wr.delta_scan_fwd(empty, empty, h0, save_states=True)
    assert out.shape == (3, 0, 40) and states.shape == (3, 0, 40) and torch.equal(hT, h0)
    _, hT = wr.delta_scan_fwd(empty, empty)
    assert torch.equal(hT, torch.zeros_like(h0))
    dx, dg, dh0 = wr.delta_scan_bwd(empty, empty, states, empty, h0)
    assert dx.shape == (3, 0, 40) and torch.equal(dh0, h0)
    x, gate, h, _, _ = inputs(3, 200, 40, BF, "sigmoid", seed=6)
    state = h.cuda()
    got = wr.delta_scan_fwd(x.cuda(), gate.cuda(), state, hT=state)
    torch.cuda.synchronize()
    assert got[1] is state
    check_fwd(got, x, gate, h, None, "sigmoid", states=False)


@pytest.mark.parametrize("form", ["sigmoid", "linear"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 33), (2, 64), (256, 512)])
def test_step_is_one_step(B, D, dtype, form):
    x, gate, h0, _, _ = inputs(B, 1, D, dtype, form, seed=B + D)
    state = h0.cuda()
    wide = torch.zeros(B, 2 * D + 1, device="cuda", dtype=dtype)
    xv = wide[:, 1:D + 1]
    xv.copy_(x[:, 0])
    out = wr.delta_scan_step(xv, gate[:, 0].cuda(), state, form=form)
    torch.cuda.synchronize()
    check_fwd((out[:, None], state), x, gate, h0, None, form, states=False)


def test_decode_continues_a_prefill():
    x, gate, h0, _, _ = inputs(2, 100, 48, F32, "sigmoid", seed=8)
    gx, gg, gh = dev(x, gate, h0)
    _, state = wr.delta_scan_fwd(gx[:, :90], gg[:, :90], gh)
    outs = [wr.delta_scan_step(gx[:, t], gg[:, t], state) for t in range(90, 100)]
    torch.cuda.synchronize()
    out, hT, _, err, _ = ref.scan(x, gate, h0)
    within(torch.stack(outs, 1), out[:, 90:], err[:, 90:] + ref.U * out[:, 90:].abs(), "out")
    within(state, hT, err[:, -1], "state")


def test_reset_stops_nan_and_inf():
    x, gate, h0, dout, dhT = inputs(1, 150, 64, F32, "linear", seed=11)
    x[0, 40, :10], x[0, 50, 10:20] = float("nan"), float("inf")
    gate[0, 64] = 0.0
    got = wr.delta_scan_fwd(x.cuda(), gate.cuda(), h0.cuda(), form="linear")
    torch.cuda.synchronize()
    clean = x.clone()
    clean[:, :64] = 0
    out, hT, _, err, _ = ref.scan(clean, gate, h0, None, "linear")
    within(got[0][:, 64:], out[:, 64:], err[:, 64:] + ref.U * out[:, 64:].abs(), "after the reset")
    assert torch.isnan(got[0][0, 41:64, :10]).all() and torch.isinf(got[0][0, 50:64, 10:20]).all()


def test_gradient_against_differences_of_the_kernel():
    # the recurrence is linear in x and h0, so a difference over any span is
    # its derivative, up to the roundings of the two sums
    x, gate, h0, dout, dhT = inputs(2, 300, 64, F32, "sigmoid", seed=12)
    gx, gg, gh, gd, gt = dev(x, gate, h0, dout, dhT)
    _, _, states = wr.delta_scan_fwd(gx, gg, gh, save_states=True)
    dx, _, dh0 = wr.delta_scan_bwd(gx, gg, states, gd, gt)
    v, w = torch.randn_like(gx), torch.randn_like(gh)
    loss = lambda o, h: (o.double() * gd).sum() + (h.double() * gt).sum()
    hi = loss(*wr.delta_scan_fwd(gx + v, gg, gh + w))
    lo = loss(*wr.delta_scan_fwd(gx - v, gg, gh - w))
    num, ana = (hi - lo) / 2, (dx.double() * v).sum() + (dh0.double() * w).sum()
    # 39040 terms of size ~1 with independent float32 errors of ~1e-6: about 1e-3
    assert abs(num - ana) <= 1e-2


def test_side_stream_and_graph():
    x, gate, h0, dout, dhT = inputs(2, 300, 128, BF, "sigmoid", seed=13)
    gx, gg, gh, gd, gt = dev(x, gate, h0, dout, dhT)
    want = wr.delta_scan_fwd(gx, gg, gh, save_states=True)
    wgrad = wr.delta_scan_bwd(gx, gg, want[2], gd, gt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wr.delta_scan_fwd(gx, gg, gh, save_states=True, stream=side)
    side.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wr.delta_scan_fwd(gx, gg, gh, save_states=True)
        grads = wr.delta_scan_bwd(gx, gg, out[2], gd, gt)
    for t in (*out, *grads):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((*out, *grads), (*want, *wgrad)):
        assert torch.equal(p, q)
    wr.delta_check_device()


def test_offsets_past_32_bits():
    # 2^31 elements and more between the first and the last row of a strided view
    T, D, gap = 3, 64, (1 << 31) + 64
    free, _ = torch.cuda.mem_get_info()
    assert free > 12 << 30
    pool = torch.empty(gap + T * D, device="cuda", dtype=BF)
    xv = torch.as_strided(pool, (2, T, D), (gap, D, 1))
    x, gate, h0, _, _ = inputs(2, T, D, BF, "sigmoid", seed=14)
    xv.copy_(x)
    got = wr.delta_scan_fwd(xv, gate.cuda(), h0.cuda(), save_states=True)
    torch.cuda.synchronize()
    check_fwd(got, x, gate, h0, None, "sigmoid")
