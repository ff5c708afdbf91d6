"""Two residual blocks of a recurrent language model on this package's kernels.

ScanBlock   norm -> projection -> gated scan -> projection + residual, with its
            gradients, and a decode step; in 8 bits too
DeltaBlock  the same around the Gated DeltaNet mixer (prefill and decode)

Run as a program it trains a ScanBlock for a few steps towards a leaky sum, then
prefills and decodes through both blocks and compares decoding with prefill.

    python examples/hybrid_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_rnn_gb300 as wr  # noqa: E402

BF = torch.bfloat16


def _normal(gen, *shape, scale):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(BF)


def quantise(w):
    """A weight's rows in e4m3, with a scale for each."""
    scale = w.float().abs().amax(-1).clamp_min(1e-12) / 448.0
    return (w.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


class ScanBlock:
    """out = stream + W_out scan(W_in norm(stream)); the stream arrives as a sum
    (``branch`` + ``stream``), as it leaves the block before.  `width`: of the
    stream, `inner`: channels of the recurrence."""

    def __init__(self, width, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.inner = inner
        self.norm = torch.ones(width, device="cuda")
        self.w_in = _normal(gen, 2 * inner, width, scale=width ** -0.5)
        self.b_in = torch.zeros(2 * inner, device="cuda")
        self.b_in[inner:] = 2.0  # decays start near 0.88
        self.w_out = _normal(gen, width, inner, scale=inner ** -0.5)
        self.kept = None

    def forward(self, branch, stream, state=None, lengths=None, train=False):
        """branch, stream [B, T, width]; returns the new stream and the state."""
        y, total, rstd = wr.delta_add_rmsnorm_fwd(branch, self.norm, stream)
        xg = wr.delta_linear_fwd(y, self.w_in, self.b_in)
        x, gate = xg[..., :self.inner], xg[..., self.inner:]  # slices, not copies
        got = wr.delta_scan_fwd(x, gate, state, lengths=lengths, save_states=train)
        out = wr.delta_linear_fwd(got[0], self.w_out, None, total)
        if train:
            self.kept = (y, total, rstd, x, gate, got[0], got[2], lengths)
        return out, got[1]

    def backward(self, dout):
        """Gradients of the last ``forward(train=True)``: of the stream (branch
        and stream alike), and of the weights by name."""
        y, total, rstd, x, gate, h, states, lengths = self.kept
        dh, dw_out, _ = wr.delta_linear_bwd(h, self.w_out, dout, want=(True, True, False))
        dx, dgate, _ = wr.delta_scan_bwd(x, gate, states, dh, lengths=lengths)
        dy, dw_in, db_in = wr.delta_linear_bwd(y, self.w_in, torch.cat([dx, dgate], -1))
        dstream, dnorm = wr.delta_add_rmsnorm_bwd(dy, total, self.norm, rstd, dout)
        return dstream, {"norm": dnorm, "w_in": dw_in, "b_in": db_in, "w_out": dw_out}

    def step(self, branch, stream, state):
        """One token, [B, width]; the state is updated in place."""
        y, total, _ = wr.delta_add_rmsnorm_fwd(branch, self.norm, stream)
        xg = wr.delta_linear_fwd(y, self.w_in, self.b_in)
        h = wr.delta_scan_step(xg[:, :self.inner], xg[:, self.inner:], state)
        return wr.delta_linear_fwd(h, self.w_out, None, total)

    def quantise(self):
        self.q_in = quantise(self.w_in)

    def step_quant(self, branch, stream, state):
        """The same with the norm's output and the first projection in 8 bits."""
        y, scale, total = wr.delta_add_rmsnorm_quant(branch, self.norm, stream)
        xg = wr.delta_linear_quant(y, scale, *self.q_in, self.b_in)
        h = wr.delta_scan_step(xg[:, :self.inner], xg[:, self.inner:], state)
        return wr.delta_linear_fwd(h, self.w_out, None, total)


class DeltaBlock:
    """The same around the gated delta rule: q, k, v, beta and the gate come from
    one projection, SiLU and the L2 norm of q and k from the mixer's prologue."""

    def __init__(self, width, heads, seed=1, d=128):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.d = heads, d
        self.norm = torch.ones(width, device="cuda")
        self.w_qkv = _normal(gen, 3 * heads * d, width, scale=width ** -0.5)
        self.w_bg = _normal(gen, 2 * heads, width, scale=width ** -0.5)
        self.b_bg = torch.cat([torch.zeros(heads), torch.full((heads,), 3.0)]).cuda()
        self.w_out = _normal(gen, width, heads * d, scale=(heads * d) ** -0.5)

    def _mixer_inputs(self, y):
        shape = y.shape[:-1] + (self.heads, self.d)
        qkv = wr.delta_linear_fwd(y, self.w_qkv).split(self.heads * self.d, -1)
        q, k, v = (t.contiguous().view(shape) for t in qkv)
        beta, gate = wr.delta_linear_fwd(y, self.w_bg, self.b_bg).float().split(self.heads, -1)
        return q, k, v, beta.contiguous(), torch.sigmoid(gate).contiguous()

    def forward(self, branch, stream, state=None):
        y, total, _ = wr.delta_add_rmsnorm_fwd(branch, self.norm, stream)
        out, state = wr.delta_fwd_prologue(*self._mixer_inputs(y), state)
        return wr.delta_linear_fwd(out.flatten(-2), self.w_out, None, total), state

    def step(self, branch, stream, state):
        y, total, _ = wr.delta_add_rmsnorm_fwd(branch, self.norm, stream)
        q, k, v, beta, gate = self._mixer_inputs(y)
        out = wr.delta_step_prologue(q, k[:, None], v[:, None], beta[:, None], gate, state)
        return wr.delta_linear_fwd(out.flatten(-2), self.w_out, None, total)


def train(steps=150, width=128, inner=256, seed=3, rate=0.005):
    """Least squares towards a leaky sum of the inputs; returns the losses."""
    block = ScanBlock(width, inner, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    masters = {n: getattr(block, n).float() for n in ("norm", "w_in", "b_in", "w_out")}
    losses, leak = [], torch.tensor(0.8, device="cuda")
    for _ in range(steps):
        x = torch.randn(8, 64, width, generator=gen, device="cuda").to(BF)
        target, _ = wr.delta_scan_fwd(x, leak.expand(x.shape).contiguous(), form="linear")
        out, _ = block.forward(x, torch.zeros_like(x), train=True)
        diff = out.float() - target.float()
        losses.append(diff.square().mean().item())
        _, grads = block.backward((2.0 * diff / diff.numel()).to(BF))
        for name, master in masters.items():
            g = grads[name].float()
            master -= rate * g / (g.square().mean().sqrt() + 1e-12)  # normalised descent
            setattr(block, name, master.to(getattr(block, name).dtype))
    return losses


def main():
    losses = train()
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    B, T, width = 2, 70, 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(B, T, width, generator=gen, device="cuda").to(BF)
    zero = torch.zeros_like(x)
    scan, delta = ScanBlock(width, 512), DeltaBlock(width, 2)
    scan.quantise()
    head, nothing = x[:, :-1].contiguous(), zero[:, :-1].contiguous()
    a, s1 = scan.forward(head, nothing)
    _, s2 = delta.forward(a, nothing)
    whole = delta.forward(scan.forward(x, zero)[0], zero)[0][:, -1]
    q1, q2 = s1.clone(), s2.clone()
    last = delta.step(scan.step(x[:, -1], zero[:, -1], s1), zero[:, -1], s2)
    last8 = delta.step(scan.step_quant(x[:, -1], zero[:, -1], q1), zero[:, -1], q2)
    rel = lambda p, q: ((p.float() - q.float()).norm() / q.float().norm()).item()
    print(f"decode against prefill: {rel(last, whole):.1e}, with 8 bits {rel(last8, whole):.1e}")
    wr.delta_check_device()
    return losses, rel(last, whole), rel(last8, whole)


if __name__ == "__main__":
    main()
