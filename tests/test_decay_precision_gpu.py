"""Decay attention after many chunks, whole or cut: the norm of the error against 64 bits.

float32: a term is off by 2^-22 at most for the tf32 products that are left out.  Sums of
8 terms are cut off by the matrix instructions, 2^-24 of the running sum on average, and a
running sum of n random terms is (i/n)^1/2 of itself on its way: 2/3 of 8 to 32 additions
for G, Q S and P V each, which add as squares where they are independent and are below 2^-21
in all up to 128 channels, with the chunks' folds (those that a state remembers, 16 of 32
tokens) 2^-24 each at random: 2^-20.  Twice that for 256 channels.

bfloat16 on the tensor cores: a token's way into the state is rounded to 2^-16; out has its
own rounding and that of P and S, each at random within half a step, sqrt(1/3) of it.
bfloat16 off them: out's own rounding alone; the state as in float32."""
import pytest
import torch

import weight_rnn_gb300 as wr
from block_ref import HALF
from test_decay_gpu import on_tc

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CHUNK = 256


def attend(q, k, v, g, h0):
    """[T, d] of one head in 64 bits, over chunks: out and the last state"""
    T, S, out = q.shape[0], h0, []
    i = torch.arange(CHUNK, device=q.device, dtype=torch.float64)
    within = torch.where(i[:, None] >= i, g ** (i[:, None] - i).clamp(min=0), 0.0)
    for t in range(0, T, CHUNK):
        a, b, c = q[t:t + CHUNK], k[t:t + CHUNK], v[t:t + CHUNK]
        n = a.shape[0]
        out.append(((a @ b.T) * within[:n, :n]) @ c + g ** (i[:n, None] + 1) * (a @ S))
        S = g ** n * S + (b * g ** (n - 1 - i[:n, None])).T @ c
    return torch.cat(out), S


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("B,T,H,dk,dv,dtype", [
    (1, 65536, 4, 128, 128, BF), (1, 20000, 8, 64, 64, BF),  # cut
    (1, 20000, 160, 64, 64, BF),                              # whole, heads shared out
    (1, 3001, 1, 256, 256, BF), (2, 5000, 2, 136, 40, BF),    # off the tensor cores, cut
    (1, 65536, 4, 64, 64, F32), (1, 9001, 2, 128, 96, F32), (1, 3001, 1, 256, 256, F32),
    (1, 6000, 320, 32, 32, F32)], ids=str)                    # (the last whole)
def test_after_many_chunks(B, T, H, dk, dv, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = (r(B, T, H, d).to(dtype) for d in (dk, dk, dv, dv))
    h0, dh = r(B, H, dk, dv), r(B, H, dk, dv)
    decay = torch.tensor([1 - 2.0 ** -9, 0.5, 1 - 2.0 ** -5], device="cuda")[torch.arange(H) % 3]
    scale = 0.3
    tc = on_tc(q, k, v)
    out, hT = wr.delta_decay_fwd(q, k, v, decay, h0, scale=scale)
    grads = wr.delta_decay_bwd(q, k, v, decay, do, h0, dh, scale=scale)
    wr.delta_check_device()
    f32 = 2.0 ** -20 if max(dk, dv) <= 128 else 2.0 ** -19
    state = 2.0 ** -16 if tc else f32
    half = HALF[BF] if dtype == BF else 0.0
    each = half * (2 / 3 if tc else 1 / 3) ** 0.5 + f32
    for b, h in [(0, 0), (B - 1, H - 1)] + ([(0, 1), (B - 1, 2)] if H > 2 else []):
        Q, K, V, D = (t[b, :, h].double() for t in (q, k, v, do))
        g, s0, sT = decay[h].double(), h0[b, h].double(), dh[b, h].double()
        o, S = attend(Q, K, V, g, s0)
        dq = attend(D, V, K, g, s0.T)[0]
        back = [t.flip(0) for t in (Q, K, V, D)]
        dv_, R = attend(back[1], scale * back[0], back[3], g, sT / g)
        dk_ = attend(back[2], back[3], scale * back[0], g, sT.T / g)[0]
        for name, got, want, most in (
                ("out", out[b, :, h], scale * o, each), ("hT", hT[b, h], S, state), ("dq", grads[0][b, :, h], scale * dq, each),
                ("dk", grads[1][b, :, h], dk_.flip(0), each), ("dv", grads[2][b, :, h], dv_.flip(0), each),
                ("dh0", grads[3][b, h], g * R, state)):
            assert rel(got, want) <= most, (name, b, h, rel(got, want), most)
            tail = slice(-300, None)  # and far into the row by itself
            if name not in ("hT", "dh0"):
                assert rel(got[tail], want[tail]) <= 1.1 * most, (name, b, h, "tail")
