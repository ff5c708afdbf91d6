"""Plain 64-bit definition of linear attention with a decay for each head, token by
token, with running bounds on what the kernels' roundings may add, for the tests."""
import torch

from block_ref import HALF, U

BF = HALF[torch.bfloat16]


def rows(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def forward(q, k, v, decay, h0=None, scale=1.0, lengths=None):
    """out, hT, and the same with every term's magnitude in its place."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = rows(lengths, B, T)
    g = decay.double()[:, None, None]
    out, big = (torch.zeros(B, T, H, dv, dtype=torch.float64) for _ in range(2))
    hT, hbig = (torch.zeros(B, H, dk, dv, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if h0 is None else h0[b].double()
        A = S.abs()
        for t in range(n[b]):
            x, y = k[b, t].double()[..., None], v[b, t].double()[:, None]
            S, A = g * S + x * y, g * A + x.abs() * y.abs()
            p = q[b, t].double()[:, None]
            out[b, t], big[b, t] = scale * (p @ S)[:, 0], abs(scale) * (p.abs() @ A)[:, 0]
        hT[b], hbig[b] = S, A
    return out, hT, big, hbig


def backward(q, k, v, decay, dout, h0=None, dhT=None, scale=1.0, lengths=None):
    """(dq, dk, dv, dh0) and the same with every term's magnitude in its place."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = rows(lengths, B, T)
    g = decay.double()[:, None, None]
    got = [torch.zeros(B, T, H, d, dtype=torch.float64) for d in (dk, dk, dv)]
    big = [torch.zeros_like(t) for t in got]
    dh0, hbig = (torch.zeros(B, H, dk, dv, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if h0 is None else h0[b].double()
        R = torch.zeros(H, dk, dv, dtype=torch.float64) if dhT is None else dhT[b].double()
        A, C = S.abs(), R.abs()
        for t in range(n[b]):
            x, y, d = k[b, t].double()[..., None], v[b, t].double()[:, None], dout[b, t].double()[..., None]
            S, A = g * S + x * y, g * A + x.abs() * y.abs()
            got[0][b, t], big[0][b, t] = scale * (S @ d)[..., 0], abs(scale) * (A @ d.abs())[..., 0]
        for t in range(n[b] - 1, -1, -1):
            p, d = q[b, t].double()[..., None], dout[b, t].double()[:, None]
            R, C = R + scale * p * d, C + abs(scale) * p.abs() * d.abs()
            x, y = k[b, t].double()[:, None], v[b, t].double()[..., None]
            got[1][b, t], big[1][b, t] = (R @ y)[..., 0], (C @ y.abs())[..., 0]
            got[2][b, t], big[2][b, t] = (x @ R)[:, 0], (x.abs() @ C)[:, 0]
            R, C = g * R, g * C
        dh0[b], hbig[b] = R, C
    return (*got, dh0), (*big, hbig)


def slack(T, d, tc):
    """What float32 sums and powers of the decay add, as a share of the terms'
    magnitudes: a sum's length in U (d channels or a chunk's tokens twice over), the
    chunks' folds, and each power's own error, 2 U for the exponential, 2 U of the
    exponent (at most 150 / log2 e where the power is not 0 in float32).  On the tensor
    cores, moreover, a token's way into the state is rounded to 2^-16, twice bfloat16's
    half step."""
    return (2 * d + 256 + T / 16 + 2 + 300) * U + (BF * BF * 1.01 if tc else 0.0)


def flushed(T, h0, *pairs):
    """A power of the decay below float32's normal range counts as 0: of each of the T
    terms that a state is the sum of, and of its first value, less than 2^-126 of what it
    is without its power is lost."""
    most = lambda t: 0.0 if t is None or t.numel() == 0 else t.abs().max().item()  # noqa: E731
    size = most(h0)
    for x, y in pairs:
        size += T * most(x) * most(y)
    return 2.0 ** -126 * size


def out_error(ref, big, T, d, dtype, tc, lost=1e-38):
    """On the tensor cores P and the state that out reads are bfloat16: half a step of
    every term; then out's own rounding."""
    e = big * (slack(T, d, tc) + (BF * (1 + 2 * BF) if tc else 0.0))
    return e + HALF[dtype] * (ref.abs() + e) + lost
