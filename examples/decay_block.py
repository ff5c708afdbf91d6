"""A block of linear attention with a decay for each head, with its feed-forward half,
on this package's kernels:

    y = layer norm(stream)             q, k, v = W_qkv y
    z = layer norm by heads(decay attention(q, k, v))
    y = layer norm(stream + W_out z)   stream += W_out z + W_down (silu(W_g y) * W_u y)

with its gradients and a decode step.  Run as a program it takes a few steps of training
towards the inputs of three tokens before, then prefills, decodes from a captured step,
and compares with the prefill of all tokens.

    python examples/decay_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_rnn_gb300 as wr  # noqa: E402

BF = torch.bfloat16


class DecayBlock:
    """`width`: of the stream, `heads` of `d` channels, `inner`: of the feed-forward half.
    The stream arrives as a sum (``branch`` + ``stream``; branch may be None)."""

    WEIGHTS = ("norm", "norm_b", "w_qkv", "head", "head_b", "w_out", "norm2", "norm2_b", "w_up", "b_up", "w_down")

    def __init__(self, width, heads, inner, d=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(  # noqa: E731
            *shape, generator=gen, device="cuda").mul_(shape[-1] ** -0.5).to(BF)
        ones, zeros = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
        self.heads, self.d, self.scale = heads, d, d ** -0.5
        self.decay = 1.0 - 2.0 ** -torch.linspace(3.0, 8.0, heads, device="cuda")
        self.norm, self.norm_b = ones(width), zeros(width)
        self.w_qkv = normal(3 * heads * d, width)
        self.head, self.head_b = ones(d), zeros(d)
        self.w_out = normal(width, heads * d)
        self.norm2, self.norm2_b = ones(width), zeros(width)
        self.w_up, self.b_up = normal(2 * inner, width), zeros(2 * inner)
        self.w_down = normal(width, inner)
        self.kept = None

    def _qkv(self, y):
        qkv = wr.delta_linear_fwd(y, self.w_qkv).unflatten(-1, (3, self.heads, self.d))
        return qkv.unbind(-3)  # slices, not copies

    def forward(self, branch, stream, state=None, lengths=None, train=False):
        """stream [B, T, width]; returns the new stream and the state [B, heads, d, d]."""
        y, s1, m1, r1 = wr.delta_add_layernorm_fwd(stream, self.norm, self.norm_b, branch)
        q, k, v = self._qkv(y)
        o, last = wr.delta_decay_fwd(q, k, v, self.decay, state, scale=self.scale, lengths=lengths)
        z, _, mo, ro = wr.delta_add_layernorm_fwd(o, self.head, self.head_b)
        a = wr.delta_linear_fwd(z.flatten(-2), self.w_out)
        y2, s2, m2, r2 = wr.delta_add_layernorm_fwd(a, self.norm2, self.norm2_b, s1)
        if train:
            f, pre = wr.delta_glu_fwd(y2, self.w_up, self.b_up, save_pre=True)
            self.kept = (y, s1, m1, r1, q, k, v, state, lengths, o, z, mo, ro, y2, s2, m2, r2, f, pre)
        else:
            f = wr.delta_glu_fwd(y2, self.w_up, self.b_up)
        return wr.delta_linear_fwd(f, self.w_down, None, s2), last

    def backward(self, dout):
        """Gradients of the last ``forward(train=True)``: of the stream (branch and stream
        alike), of the state that it began with, and of the weights by name."""
        y, s1, m1, r1, q, k, v, state, lengths, o, z, mo, ro, y2, s2, m2, r2, f, pre = self.kept
        df, dw_down, _ = wr.delta_linear_bwd(f, self.w_down, dout, want=(True, True, False))
        dy2, dw_up, db_up = wr.delta_glu_bwd(y2, self.w_up, df, pre)
        da, dnorm2, dnorm2_b = wr.delta_add_layernorm_bwd(dy2, s2, self.norm2, m2, r2, dout)
        dz, dw_out, _ = wr.delta_linear_bwd(z.flatten(-2), self.w_out, da, want=(True, True, False))
        do, dhead, dhead_b = wr.delta_add_layernorm_bwd(dz.view(o.shape), o, self.head, mo, ro)
        dq, dk, dv, dstate = wr.delta_decay_bwd(q, k, v, self.decay, do, state, scale=self.scale, lengths=lengths)
        dqkv = torch.stack([dq, dk, dv], -3).flatten(-3)
        dy, dw_qkv, _ = wr.delta_linear_bwd(y, self.w_qkv, dqkv, want=(True, True, False))
        dstream, dnorm, dnorm_b = wr.delta_add_layernorm_bwd(dy, s1, self.norm, m1, r1, da)
        grads = (dnorm, dnorm_b, dw_qkv, dhead, dhead_b, dw_out, dnorm2, dnorm2_b, dw_up, db_up, dw_down)
        return dstream, dstate, dict(zip(self.WEIGHTS, grads))

    def step(self, branch, stream, state):
        """One token, [B, width]; the state is updated in place."""
        y, s1, _, _ = wr.delta_add_layernorm_fwd(stream, self.norm, self.norm_b, branch)
        o = wr.delta_decay_step(*self._qkv(y), self.decay, state, scale=self.scale)
        z = wr.delta_add_layernorm_fwd(o, self.head, self.head_b)[0]
        a = wr.delta_linear_fwd(z.flatten(-2), self.w_out)
        y2, s2, _, _ = wr.delta_add_layernorm_fwd(a, self.norm2, self.norm2_b, s1)
        return wr.delta_linear_fwd(wr.delta_glu_fwd(y2, self.w_up, self.b_up), self.w_down, None, s2)


def train(steps=20, width=128, seed=3, rate=0.002):
    """Least squares towards the tokens of three steps before; returns the losses."""
    block = DecayBlock(width, 2, 192, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    masters = {n: getattr(block, n).float() for n in block.WEIGHTS}
    losses = []
    for _ in range(steps):
        x = torch.randn(8, 64, width, generator=gen, device="cuda").to(BF)
        out, _ = block.forward(None, x, train=True)
        diff = out.float()
        diff[:, 3:] -= x[:, :-3].float()
        losses.append(diff.square().mean())
        _, _, grads = block.backward((2.0 * diff / diff.numel()).to(BF))
        for name, master in masters.items():
            g = grads[name].float()
            master -= rate * g / (g.square().mean().sqrt() + 1e-12)  # normalised descent
            setattr(block, name, master.to(getattr(block, name).dtype))
    return torch.stack(losses).tolist()


def decode(block, x, state):
    """x [B, n, width] token by token through a step captured once; the last one's output."""
    token, s = x[:, 0].contiguous(), state.clone()
    block.step(None, token, s.clone())  # kernels are loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.step(None, token, s)
    for t in range(x.shape[1]):
        token.copy_(x[:, t])
        graph.replay()
    return out, s


def main():
    losses = train()
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    B, T, new, width = 2, 200, 6, 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(B, T + new, width, generator=gen, device="cuda").to(BF)
    block = DecayBlock(width, 4, 512)
    whole, end = block.forward(None, x)
    _, state = block.forward(None, x[:, :T].contiguous())
    last, state = decode(block, x[:, T:], state)
    rel = lambda p, q: ((p.float() - q.float()).norm() / q.float().norm()).item()  # noqa: E731
    off = rel(last, whole[:, -1]), rel(state, end)
    print(f"decode against prefill: {off[0]:.1e}, states {off[1]:.1e}")
    wr.delta_check_device()
    return losses, off


if __name__ == "__main__":
    main()
