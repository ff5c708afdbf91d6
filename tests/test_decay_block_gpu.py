"""Layer norm, decay attention and the gated feed-forward layer run together, as a block
uses them (examples/decay_block.py): gradients against float64 autograd of the same
formulas, decoding against prefill, eager and captured steps."""
import importlib.util
import os

import pytest
import torch

import decay_ref
from block_ref import HALF, act

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# Every rounding to bfloat16 is within half a step, 2^-8, of what it rounds, and they are
# independent, so that they add as squares, times the powers in which what they round
# enters the output.  Forward: the first norm's output enters q, k and v (3), which are
# rounded themselves (1, 1, 1), as are P and S (1 together), the attention's output, the
# head norm's, the projection's and the second norm's (1 each); all of that enters both
# halves of the gated layer (2); its output and the stream are rounded (1, 1):
# (4 (9 + 3 + 1 + 4) + 2)^(1/2) = 8.4.
STEPS = 8.4 * HALF[torch.bfloat16]
# The gradients take as many roundings on the way back, and read what the way forth rounded.
STEPS_BACK = 2.0 ** 0.5 * 2 * STEPS


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decay_block", os.path.join(ROOT, "examples", "decay_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return ((a.detach().cpu().double() - b).norm() / b.norm()).item()


def layer_norm(t, w, b):
    d = t - t.mean(-1, keepdim=True)
    return d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w + b


def attention(q, k, v, decay, h0, scale, n):
    """in one piece: weights g^(t-j), and g^(t+1) for the state before; rows of n tokens"""
    B, T, H, d = q.shape
    t = torch.arange(T, dtype=torch.float64)
    apart = t[:, None] - t
    w = torch.where(apart >= 0, decay[:, None, None] ** apart.clamp(min=0), 0.0)
    out = torch.einsum("bthd,bjhd,htj,bjhe->bthe", q, k, w, v)
    out = out + torch.einsum("bthd,bhde,th->bthe", q, h0, decay ** (t[:, None] + 1))
    return scale * torch.where(t[None, :, None, None] < n[:, None, None, None], out, 0.0)


def test_block_gradients(example):
    B, T, width, heads, inner, d = 3, 150, 96, 2, 136, 32
    block = example.DecayBlock(width, heads, inner, d, seed=2)
    gen = torch.Generator().manual_seed(1)
    normal = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731
    for name in ("norm", "norm_b", "head", "head_b", "norm2", "norm2_b", "b_up"):
        t = getattr(block, name)
        t += 0.2 * normal(*t.shape).cuda()
    x, stream, dout = (normal(B, T, width).to(torch.bfloat16) for _ in range(3))
    state = normal(B, heads, d, d)
    n = torch.tensor([150, 33, 129], dtype=torch.int32)
    out, _ = block.forward(x.cuda(), stream.cuda(), state.cuda(), lengths=n.cuda(), train=True)
    dstream, dstate, grads = block.backward(dout.cuda())
    torch.cuda.synchronize()

    p = {name: getattr(block, name).detach().cpu().double().requires_grad_(True) for name in block.WEIGHTS}
    s = (x.double() + stream.double()).requires_grad_(True)
    h0 = state.double().requires_grad_(True)
    q, k, v = (layer_norm(s, p["norm"], p["norm_b"]) @ p["w_qkv"].T).unflatten(-1, (3, heads, d)).unbind(-3)
    o = attention(q, k, v, block.decay.cpu().double(), h0, block.scale, n)
    s2 = s + layer_norm(o, p["head"], p["head_b"]).flatten(-2) @ p["w_out"].T
    g, u = (layer_norm(s2, p["norm2"], p["norm2_b"]) @ p["w_up"].T + p["b_up"]).chunk(2, -1)
    want = (act("silu", g) * u) @ p["w_down"].T + s2
    want.backward(dout.double())
    assert rel(out, want.detach()) <= STEPS
    assert rel(dstream, s.grad) <= STEPS_BACK
    assert rel(dstate, h0.grad) <= STEPS_BACK
    for name, got in grads.items():
        assert rel(got, p[name].grad) <= STEPS_BACK, name


def test_attention_in_one_piece_is_the_recurrence():
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(2, 40, 3, 8, generator=gen) for _ in range(3))
    decay, h0 = torch.tensor([0.5, 0.9, 1.0]), torch.randn(2, 3, 8, 8, generator=gen)
    n = torch.tensor([40, 17])
    got = attention(*(t.double() for t in (q, k, v, decay, h0)), 0.3, n)
    want = decay_ref.forward(q, k, v, decay, h0, 0.3, n)[0]
    assert (got - want).abs().max() <= 1e-12 * want.abs().max()


def test_captured_steps_are_the_eager_ones(example):
    block = example.DecayBlock(96, 3, 200, 32, seed=6)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5, 4, 96, generator=gen, device="cuda").to(torch.bfloat16)
    state = torch.randn(5, 3, 32, 32, generator=gen, device="cuda")
    out, last = example.decode(block, x, state)
    for t in range(4):
        want = block.step(None, x[:, t].contiguous(), state)
    assert torch.equal(out, want) and torch.equal(last, state)


def test_example_runs(example):
    losses, (out, state) = example.main()
    assert all(loss == loss and loss < float("inf") for loss in losses)
    assert out <= 2 ** 0.5 * STEPS  # both ways have their roundings
    assert state <= 2 ** 0.5 * STEPS
