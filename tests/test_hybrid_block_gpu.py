"""The example's blocks: gradients of a ScanBlock against float64 autograd of the
same formulas, decoding against prefill, and a training run that learns."""
import importlib.util
import os

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_block", os.path.join(ROOT, "examples", "hybrid_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return ((a.detach().cpu().double() - b).norm() / b.norm()).item()


def test_scan_block_gradients(example):
    B, T, width, inner = 3, 90, 64, 96
    block = example.ScanBlock(width, inner, seed=2)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(B, T, width, generator=gen).to(torch.bfloat16)
    stream = torch.randn(B, T, width, generator=gen).to(torch.bfloat16)
    dout = torch.randn(B, T, width, generator=gen).to(torch.bfloat16)
    lengths = torch.tensor([90, 33, 64], dtype=torch.int32)
    out, _ = block.forward(x.cuda(), stream.cuda(), lengths=lengths.cuda(), train=True)
    dstream, grads = block.backward(dout.cuda())
    torch.cuda.synchronize()

    p = {n: getattr(block, n).detach().cpu().double().requires_grad_(True)
         for n in ("norm", "w_in", "b_in", "w_out")}
    s = (x.double() + stream.double()).requires_grad_(True)
    _, _, y = ref.norm(s, None, p["norm"], 1e-6)
    xg = y @ p["w_in"].T + p["b_in"]
    h, _, _, _, _ = ref.scan(xg[..., :inner], xg[..., inner:], None, lengths, "sigmoid")
    want = h @ p["w_out"].T + s
    want.backward(dout.double())
    # five roundings to bfloat16 lie between the ends, each within half a step,
    # 2^-8, of what passes it
    tol = 5 * 2.0 ** -8
    assert rel(out, want.detach()) <= tol
    assert rel(dstream, s.grad) <= tol
    for n, g in grads.items():
        assert rel(g, p[n].grad) <= tol, n


def test_example_runs(example):
    losses, decode, decode8 = example.main()
    assert losses[-1] < 0.8 * losses[0]
    # two blocks, each with four bfloat16 roundings of what it adds
    assert decode <= 8 * 2.0 ** -8
    # and operands in e4m3: half a step is 2^-4 of each term, independent terms
    assert decode8 <= 2.0 ** -4 + 8 * 2.0 ** -8
