"""Linear attention with a decay for each head against its 64-bit definition."""
import pytest
import torch

import decay_ref as ref
import weight_rnn_gb300 as wr
from block_ref import U, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, H, dk, dv, dtype, seed=0, layout="fused"):
    gen = torch.Generator().manual_seed(1000 + seed)
    if layout == "fused":  # slices of one projection's output
        x = torch.randn(B, T, H * (2 * dk + dv), generator=gen).to(dtype)
        q, k, v = (t.unflatten(-1, (H, -1)) for t in x.split((H * dk, H * dk, H * dv), -1))
    elif layout == "heads":  # [B, H, T, d] in memory
        q, k, v = (torch.randn(B, H, T, d, generator=gen).to(dtype).transpose(1, 2) for d in (dk, dk, dv))
    else:  # odd addresses
        q, k, v = (torch.randn(B, T, H, d + 1, generator=gen).to(dtype)[..., 1:] for d in (dk, dk, dv))
    decay = 1.0 - 2.0 ** (-1.0 - 9.0 * torch.rand(H, generator=gen))
    h0 = torch.randn(B, H, dk, dv, generator=gen)
    return q, k, v, decay, h0


def same_strides(t):
    """on the GPU with the strides that it has here"""
    base = torch.empty(0, dtype=t.dtype, device=DEV)
    to = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype, device=DEV)
    to.copy_(torch.empty(0, dtype=t.dtype).set_(t.untyped_storage(), 0, (to.numel(),)))
    return base.set_(to.untyped_storage(), t.storage_offset(), t.shape, t.stride())


def on_tc(q, k, v):
    dk, dv = q.shape[-1], v.shape[-1]
    whole = all(t.storage_offset() % 8 == 0 and (t.stride(1) > 0 or t.shape[1] == 1) and
                all(s % 8 == 0 for s, n in zip(t.stride()[:-1], t.shape) if n > 1) for t in (q, k, v))
    return q.dtype == BF and dk <= 128 and dk % 8 == 0 and dv % 8 == 0 and whole


def check(q, k, v, decay, h0, scale=0.3, lengths=None, dhT=True, seed=0, grads=True):
    B, T, H, dk = q.shape
    dv, dt, tc = v.shape[-1], q.dtype, on_tc(q, k, v)
    to = lambda t: None if t is None else same_strides(t)  # noqa: E731
    Q, K, V, G, H0, L = (to(t) for t in (q, k, v, decay, h0, lengths))
    out, hT = wr.delta_decay_fwd(Q, K, V, G, H0, scale=scale, lengths=L)
    clean = [t.clone() for t in (q, k, v)]
    for b, n in enumerate(ref.rows(lengths, B, T)):  # what later tokens hold does not matter
        for t in clean:
            t[b, n:] = 0
    ro, rh, bo, bh = ref.forward(*clean, decay, h0, scale, lengths)
    lost = ref.flushed(T, h0, (clean[1], clean[2]))
    top = lambda t: max(1.0, t.abs().max().item() if t.numel() else 0.0)  # noqa: E731
    # on the tensor cores out reads no less than 2^-64 of the state before its chunk
    read = 2.0 ** 62 if tc else 1.0
    within(out, ro, ref.out_error(ro, bo, T, dk, dt, tc, read * lost * max(1.0, abs(scale)) * dk * top(clean[0])), "out")
    within(hT, rh, bh * ref.slack(T, 1, tc) + lost, "hT")
    if grads:
        gen = torch.Generator().manual_seed(2000 + seed)
        do = torch.randn(B, T, H, dv, generator=gen).to(dt)
        dh = torch.randn(B, H, dk, dv, generator=gen) if dhT else None
        got = wr.delta_decay_bwd(Q, K, V, G, do.to(DEV), H0, to(dh), scale=scale, lengths=L)
        for b, n in enumerate(ref.rows(lengths, B, T)):
            do[b, n:] = 0
        rg, bg = ref.backward(*clean, decay, do, h0, dh, scale, lengths)
        lost = max(lost, ref.flushed(T, dh, (clean[0], do))) * max(1.0, abs(scale))
        for name, g, r, m in zip(("dq", "dk", "dv"), got, rg, bg):
            least = read * lost * (dk + dv) * max(top(t) for t in (*clean, do))
            within(g, r, ref.out_error(r, m, T, max(dk, dv), dt, tc, least), name)
        within(got[3], rg[3], bg[3] * ref.slack(T, 1, tc) + lost, "dh0")
    wr.delta_check_device()
    return out, hT


SHAPES = [  # B, T, H, dk, dv
    (1, 1, 1, 128, 128), (2, 2, 3, 64, 64), (1, 127, 2, 128, 128), (1, 128, 1, 128, 128), (2, 129, 2, 128, 64),
    (1, 300, 3, 80, 48), (3, 70, 2, 16, 24), (1, 257, 1, 8, 8), (1, 200, 2, 128, 200), (2, 391, 1, 40, 136),
    (1, 140, 1, 104, 256),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    check(*inputs(*shape, dtype, seed=shape[1]), seed=shape[1])


@pytest.mark.parametrize("shape", [(2, 45, 2, 3, 5), (1, 70, 1, 1, 1), (1, 40, 1, 256, 256), (1, 131, 2, 100, 60),
                                   (1, 66, 1, 130, 70)], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_dims_without_the_tensor_cores(shape, dtype):
    q, k, v, decay, h0 = inputs(*shape, dtype)
    assert not on_tc(q, k, v)
    check(q, k, v, decay, h0)


@pytest.mark.parametrize("layout", ["heads", "odd"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_layouts(layout, dtype):
    check(*inputs(2, 150, 3, 64, 32, dtype, layout=layout))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("what", ["heads of k and v", "rows of q", "rows of k, heads of v", "tokens"])
def test_shared_heads_rows_and_tokens(what, dtype):
    """Axes with a stride of 0; a gradient is that of each place by itself."""
    B, T, H = 3, 150, 4
    q, k, v, decay, h0 = inputs(B, T, H, 64, 48, dtype, layout="heads")
    wide = lambda t: t.expand(B, T, H, t.shape[-1])  # noqa: E731
    if what == "heads of k and v":
        k, v = wide(k[:, :, 1:2]), wide(v[:, :, 2:3])
    elif what == "rows of q":
        q = wide(q[1:2])
    elif what == "rows of k, heads of v":
        k, v = wide(k[2:]), wide(v[:, :, :1])
    else:
        v = wide(v[:, 7:8])
    check(q, k, v, decay, h0, lengths=torch.tensor([150, 0, 129], dtype=torch.int32))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_lengths_and_what_lies_past_them(dtype):
    lengths = torch.tensor([0, 1, 128, 129, 260, 300, 999, -4], dtype=torch.int32)
    q, k, v, decay, h0 = inputs(8, 300, 2, 64, 48, dtype)
    for b, n in enumerate(ref.rows(lengths, 8, 300)):
        for t, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
            t[b, n:] = bad
    check(q, k, v, decay, h0, lengths=lengths)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_ends_of_the_decays_range(dtype):
    q, k, v, _, h0 = inputs(1, 300, 8, 32, 32, dtype)
    decay = torch.tensor([0.0, 1.0, 1e-38, 1e-30, 1e-3, 0.3, 0.7, 1.0 - 2.0 ** -24])
    check(q, k, v, decay, h0)


def test_large_values_under_strong_decays():
    """A row's products pass over its least power of the decay on their way, and stay in
    float32's range."""
    q, k, v, _, h0 = inputs(1, 300, 6, 64, 32, BF)
    decay = torch.tensor([0.0, 1e-30, 1e-3, 0.3, 0.5, 0.6])
    check(1e4 * q, 1e4 * k, 1e4 * v, decay, h0)


def test_tokens_without_values():
    """What is left of a state that is all but forgotten shows where a token has no values."""
    q, k, v, _, h0 = inputs(1, 300, 6, 64, 32, BF)
    v[:, 20:160] = 0
    check(q, k, v, torch.tensor([0.0, 1e-30, 1e-3, 0.3, 0.7, 0.9]), h0)


@pytest.mark.parametrize("scale", [0.0, -1.5, 1.0, 64.0])
def test_scales(scale):
    check(*inputs(1, 140, 2, 64, 64, BF), scale=scale)


def test_without_states():
    q, k, v, decay, _ = inputs(2, 140, 2, 64, 64, BF)
    check(q, k, v, decay, None, dhT=False)


# one row of few heads: the time axis is cut into segments
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 2100, 1, 64, 64), (2, 1500, 2, 128, 136)])
def test_segments(B, T, H, dk, dv, dtype):
    lengths = torch.tensor([T] if B == 1 else [701, 0], dtype=torch.int32)
    q, k, v, decay, h0 = inputs(B, T, H, dk, dv, dtype)
    decay[0] = 1.0  # a head that forgets nothing shows every segment's state
    if H > 1:
        decay[1] = 0.0
    check(q, k, v, decay, h0, lengths=lengths)


# more heads than the GPU has SMs: CTAs share heads and hand states over; in the gradients
# also beside one another.  160 and 51 heads, 480 and 153 with all three passes.
@pytest.mark.parametrize("B,T,H,dk,dv", [(5, 640, 32, 32, 32), (3, 389, 17, 64, 24), (2, 300, 80, 16, 136)])
def test_more_heads_than_sms(B, T, H, dk, dv):
    q, k, v, decay, h0 = inputs(B, T, H, dk, dv, BF)
    decay[0], decay[1], decay[5] = 1.0, 0.0, 1.0
    check(q, k, v, decay, h0)


def test_precision_of_states_and_outputs():
    """Over many elements the roundings are at random: the states within a tenth of the
    bound above, out within bfloat16's half step over sqrt(3) for each of its own rounding
    and that of P and S, sqrt(2) of it together."""
    q, k, v, decay, h0 = inputs(1, 600, 2, 128, 128, BF)
    out, hT = check(q, k, v, decay, h0, grads=False)
    ro, rh, _, _ = ref.forward(q, k, v, decay, h0, 0.3)
    rel = lambda a, b: ((a.cpu().double() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(hT, rh) <= 2.0 ** -16
    assert rel(out, ro) <= ref.BF * (2 / 3) ** 0.5


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 128, 128), (3, 2, 64, 96), (2, 3, 5, 7), (400, 1, 16, 40), (1, 2, 256, 256),
                                       (320, 1, 130, 33)])
def test_step(B, H, dk, dv, dtype):
    q, k, v, decay, h0 = inputs(B, 3, H, dk, dv, dtype)
    state, S = h0.to(DEV), h0
    Q, K, V = (same_strides(t) for t in (q, k, v))
    for t in range(3):
        out = wr.delta_decay_step(Q[:, t], K[:, t], V[:, t], decay.to(DEV), state, scale=0.3)
        ro, S, bo, bS = ref.forward(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], decay, S.float(), 0.3)
        within(out, ro[:, 0], ref.out_error(ro, bo, 1, dk, dtype, False)[:, 0], "out")
        within(state, S, 4 * U * bS, "state")
        S = state.cpu()  # one step at a time


def test_steps_continue_the_forward():
    q, k, v, decay, h0 = inputs(2, 200, 2, 64, 64, F32)
    Q, K, V, G = (same_strides(t) for t in (q, k, v, decay))
    want, hT = wr.delta_decay_fwd(Q, K, V, G, h0.to(DEV), scale=0.5)
    _, state = wr.delta_decay_fwd(Q[:, :190], K[:, :190], V[:, :190], G, h0.to(DEV), scale=0.5)
    for t in range(190, 200):
        out = wr.delta_decay_step(Q[:, t], K[:, t], V[:, t], G, state, scale=0.5)
        torch.testing.assert_close(out, want[:, t], rtol=1e-5, atol=1e-4)
    torch.testing.assert_close(state, hT, rtol=1e-5, atol=1e-4)


def test_no_tokens():
    q, k, v, decay, h0 = (t.to(DEV) for t in inputs(2, 0, 2, 16, 16, BF))
    out, hT = wr.delta_decay_fwd(q, k, v, decay, h0)
    assert out.shape == (2, 0, 2, 16) and torch.equal(hT, h0)
    assert torch.equal(wr.delta_decay_fwd(q, k, v, decay)[1], torch.zeros_like(h0))
    dq, dk, dv, dh0 = wr.delta_decay_bwd(q, k, v, decay, out, h0, h0)
    assert dq.shape == q.shape and torch.equal(dh0, h0)


def test_state_in_place_and_given_outputs():
    q, k, v, decay, h0 = (t.to(DEV) for t in inputs(1, 700, 2, 64, 136, BF))
    want = wr.delta_decay_fwd(q, k, v, decay, h0)
    state, out = h0.clone(), torch.empty_like(want[0])
    got = wr.delta_decay_fwd(q, k, v, decay, state, out=out, hT=state)
    assert got[0] is out and got[1] is state
    assert torch.equal(out, want[0]) and torch.equal(state, want[1])


@pytest.mark.parametrize("B,T,H", [(1, 1500, 2), (5, 400, 40)])
def test_the_same_on_a_side_stream_again_and_from_a_graph(B, T, H):
    q, k, v, decay, h0 = (t.to(DEV) for t in inputs(B, T, H, 64, 64, BF))
    do, dh = torch.randn_like(v).contiguous(), torch.randn_like(h0)
    state = h0.clone()
    step_in = [t[:, 5] for t in (q, k, v)]

    def all_of(stream=None):
        return (*wr.delta_decay_fwd(q, k, v, decay, h0, stream=stream),
                *wr.delta_decay_bwd(q, k, v, decay, do, h0, dh, stream=stream))
    want = all_of()
    wr.delta_decay_step(*step_in, decay, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, kept = torch.cuda.CUDAGraph(), h0.clone()
    with torch.cuda.graph(graph):
        captured = all_of()
        wr.delta_decay_step(*step_in, decay, kept)
    for _ in range(3):
        for t in captured:
            t.zero_()
        kept.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert torch.equal(kept, state)


def test_gradients_are_the_forwards_slopes():
    """Along a direction, in float32: (L(x + eps d) - L(x - eps d)) / 2 eps.  L is linear
    in each argument alone, so there is no truncation; float32's rounding of L's terms
    stays, a few hundred U of their magnitudes over eps."""
    q, k, v, decay, h0 = (t.to(DEV) for t in inputs(1, 150, 2, 24, 16, F32))
    gen = torch.Generator(device=DEV).manual_seed(7)
    do = torch.randn(v.shape, generator=gen, device=DEV)
    dh = torch.randn(h0.shape, generator=gen, device=DEV)
    grads = wr.delta_decay_bwd(q, k, v, decay, do, h0, dh, scale=0.3)

    def loss(*a):
        out, hT = wr.delta_decay_fwd(*a[:3], decay, a[3], scale=0.3)
        return (out.double() * do).sum() + (hT.double() * dh).sum()
    args = [q, k, v, h0]
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=gen, device=DEV)
        up, down = (list(args) for _ in range(2))
        up[i], down[i] = args[i] + d, args[i] - d
        slope = (loss(*up) - loss(*down)) / 2
        want = (g.double() * d).sum()
        size = (g.double() * d).abs().sum()
        assert abs(slope - want) <= 1e-4 * size, (i, slope.item(), want.item())


@pytest.mark.parametrize("B,T,H", [(2, 900, 3), (5, 400, 40)])
def test_calls_on_two_streams_at_once(B, T, H):
    sets = [[t.to(DEV) for t in inputs(B, T, H, 128, 128, BF, seed=s)] for s in range(2)]
    want = [wr.delta_decay_fwd(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append(wr.delta_decay_fwd(*s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[0], x[0]) and torch.equal(w[1], x[1]) for x in g)


def test_past_2_31_elements():
    B, T, H, d = 1, (1 << 19) + 130, 32, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(B, T, H, d, generator=gen, device=DEV, dtype=BF) for _ in range(3))
    assert q.numel() > 1 << 31
    decay = torch.full((H,), 0.5, device=DEV)  # 300 tokens back nothing is left in float32
    out, hT = wr.delta_decay_fwd(q, k, v, decay)
    tail = [t[:, -700:, :2].float().cpu() for t in (q, k, v)]
    ro, rh, bo, bh = ref.forward(*tail, decay[:2].cpu())
    within(out[:, -300:, :2], ro[:, -300:], ref.out_error(ro, bo, T, d, BF, True)[:, -300:], "out")
    within(hT[:, :2], rh, bh * ref.slack(T, 1, True), "hT")
    del out
    do = torch.randn(B, T, H, d, generator=gen, device=DEV, dtype=BF)
    got = wr.delta_decay_bwd(q, k, v, decay, do)
    tail.append(do[:, -700:, :2].float().cpu())
    rg, bg = ref.backward(*tail[:3], decay[:2].cpu(), tail[3])
    for name, g, r, m in zip(("dq", "dk", "dv"), got, rg, bg):
        within(g[:, -300:, :2], r[:, -300:], ref.out_error(r, m, T, d, BF, True)[:, -300:], name)
    wr.delta_check_device()
