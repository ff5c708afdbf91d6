"""The gated linear recurrence where products of its decays leave float32's
range though no state does, and where resets meet Inf and NaN: forward and
backward, on one CTA a row and in clusters, against the 64-bit definition.

Bounds are those of test_scan_gpu.py, with 2^-126 on top: below float32's normal
range a value is not held to relative accuracy."""
import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
LEAST = 2.0 ** -126


def repeated(T, *runs):
    """gates from (value, steps) runs, over and over"""
    one = torch.cat([torch.full((n,), float(v)) for v, n in runs])
    return one.repeat(-(-T // len(one)))[:T]


def at(T, base, **places):
    v = torch.full((T,), float(base)) if isinstance(base, (int, float)) else base.clone()
    for k, p in places.items():
        for i in range(int(k[1:]), T, 1000000 if k[0] == "t" else 400):
            v[i] = p
    return v


def linear_channels(T, gen):
    """(gate, x, h0, dout, dhT) a channel"""
    r = lambda: torch.randn(T, generator=gen)
    z, one = torch.zeros(T), torch.ones(T)
    e = T - 4
    burst = repeated(T, (0.9, 3), (1e4, 10), (0.0, 1), (0.9, 20))
    tiny = torch.full((T,), 1e-30)
    # down and up again, from either end
    dips = torch.cat([repeated(T, (1e-3, 14), (1e3, 14))[:(T - 14) // 28 * 28 + 14], one])[:T]
    return {
        # decays overflow over nothing, over a state that stands still, and with the offsets
        "zeros": (2 * one, z, 0.0, z, 0.0),
        "still": (2 * one, one, -1.0, one, -2.0),
        "still_high": (2 * one, one * 2.0 ** 40, -2.0 ** 40, one * 2.0 ** 40, -2.0 ** 41),
        # a reset behind gates whose product overflows, or that are no numbers
        "burst": (burst, tiny, 1e-30, tiny, 1e-30),
        "nan_gate": (at(T, 0.9, r2=NAN, r5=0.0), r(), 1.0, r(), 1.0),
        "inf_gate": (at(T, 0.9, r2=INF, r5=0.0), r(), 1.0, r(), 1.0),
        "nan_early": (at(T, 0.9, r2=NAN, r100=0.0), r(), 1.0, r(), 1.0),
        "nan_x_reset": (at(T, 0.9, r4=0.0), at(T, r(), r2=NAN), 1.0, at(T, r(), r7=NAN), 1.0),
        # nothing resets: Inf and NaN stay, however small the decays
        "nan_stays": (0.3 * one, at(T, r(), t3=NAN), 1.0, at(T, r(), **{f"t{e}": NAN}), 1.0),
        "inf_stays": (0.3 * one, at(T, r(), t3=INF), 1.0, at(T, r(), **{f"t{e}": -INF}), 1.0),
        "nan_stays_small": (1e-3 * one, at(T, r(), t3=NAN), 1.0, at(T, r(), **{f"t{e}": NAN}), 1.0),
        "inf_stays_small": (-1e-3 * one, at(T, r(), t3=INF), 1.0, at(T, r(), **{f"t{e}": INF}), 1.0),
        # a product that falls below the range and comes back, over a large state
        "dips": (dips, z, 1e20, z, 1e20),
        "decayed": (0.3 * one, z, 1e30, z, 0.0),
        "grad_decayed": (0.3 * one, z, 0.0, z, 1e30),
        # ordinary values, strong decays and a reset now and then
        "strong": (0.3 * torch.rand(T, generator=gen), r(), 1.0, r(), 1.0),
        "plain": (at(T, 0.5 + 0.5 * torch.rand(T, generator=gen), r77=0.0), r(), 1.0, r(), 1.0),
        "grows": (1.01 * one, r(), 1.0, r(), 1.0),
    }


def sigmoid_channels(T, gen):
    r = lambda: torch.randn(T, generator=gen)
    z, one = torch.zeros(T), torch.ones(T)
    return {
        "inf_stays": (-1.0 * one, at(T, r(), t3=INF), 1.0, at(T, r(), **{f"t{T - 4}": -INF}), 1.0),
        "inf_stays_small": (-8.0 * one, at(T, r(), t3=INF), 1.0, at(T, r(), **{f"t{T - 4}": INF}), 1.0),
        "nan_stays": (-8.0 * one, at(T, r(), t3=NAN), 1.0, at(T, r(), **{f"t{T - 4}": NAN}), 1.0),
        "decayed": (-1.0 * one, z, 1e30, z, 0.0),
        "grad_decayed": (-1.0 * one, z, 0.0, z, 1e30),
        "strong": (-5.0 + 3.0 * r(), r(), 1.0, r(), 1.0),
        "plain": (2.0 * r() + 2.0, r(), 1.0, r(), 1.0),
    }


def stacked(B, T, D, dtype, form, seed):
    """every channel kind over and over, each row shifted by one channel"""
    gen = torch.Generator().manual_seed(seed)
    kinds = (linear_channels if form == "linear" else sigmoid_channels)(T, gen)
    names = [list(kinds)[(c + b) % len(kinds)] for b in range(B) for c in range(D)]
    col = lambda i: torch.stack([torch.as_tensor(kinds[n][i]) for n in names])
    seq = lambda i: col(i).view(B, D, T).transpose(1, 2).contiguous()
    gate = seq(0) if form == "linear" else seq(0).to(dtype)
    return names, seq(1).to(dtype), gate, col(2).view(B, D).float(), seq(3).to(dtype), col(4).view(B, D).float()


# a CTA a row; clusters of 2 forward and 4 backward, of 8, of 16; whole rows,
# pairs and single channels
SHAPES = [(160, 300, 32), (160, 140, 31), (1, 256, 32), (1, 250, 34), (20, 1100, 32), (1, 2100, 32), (2, 2085, 33)]


@pytest.mark.parametrize("form", ["linear", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_out_of_range(shape, dtype, form):
    B, T, D = shape
    names, x, gate, h0, dout, dhT = stacked(B, T, D, dtype, form, seed=T + D)
    gx, gg, gh, gd, gt = (t.cuda() for t in (x, gate, h0, dout, dhT))
    got = wr.delta_scan_fwd(gx, gg, gh, form=form, save_states=True)
    out, hT, before, err, _ = ref.scan(x, gate, h0, None, form)
    eb = torch.cat([torch.zeros_like(err[:, :1]), err[:, :-1]], 1)
    # the backward from the definition's states: its own faults are its own
    grads = wr.delta_scan_bwd(gx, gg, before[:, ::64].float().contiguous().cuda(), gd, gt, form=form)
    torch.cuda.synchronize()
    want, gerr = ref.scan_grad(x, gate, h0, dout, dhT, None, form)
    half = ref.HALF
    checks = [("out", got[0], out, err, half[dtype]), ("hT", got[1], hT, err[:, -1], 0.0),
              ("states", got[2], before[:, ::64], eb[:, ::64], 0.0)]
    checks += [(n, g, w, e, h) for n, g, w, e, h in zip(("dx", "dgate", "dh0"), grads, want, gerr,
                                                       (half[dtype], half[gate.dtype], ref.U))]
    for what, g, w, e, h in checks:
        g = g.cpu()
        for kind in dict.fromkeys(names):
            pick = torch.tensor([n == kind for n in names]).view(B, D)
            sel = lambda t: t.transpose(1, 2)[pick] if t.dim() == 3 else t[pick]
            if kind in ("zeros", "still", "still_high"):  # every step is exact (and the bounds overflow)
                assert torch.equal(sel(g).double(), sel(w)), f"{what} of {kind}"
            else:
                ref.within(sel(g), sel(w), sel(e) + h * (sel(w).abs() + sel(e)) + LEAST, f"{what} of {kind}")


@pytest.mark.parametrize("B,T", [(160, 300), (1, 700)])
def test_ragged_rows_out_of_range(B, T):
    D = 34
    names, x, gate, h0, dout, dhT = stacked(B, T, D, F32, "linear", seed=1)
    lengths = torch.tensor([(37 * b + 131) % (T + 1) for b in range(B)], dtype=torch.int32)
    # what a row does not reach stands for its end: the gradients start there
    live = torch.arange(T)[None, :, None] < lengths[:, None, None]
    clean = lambda t: torch.where(live, t, torch.zeros_like(t))
    got = wr.delta_scan_fwd(x.cuda(), gate.cuda(), h0.cuda(), form="linear", lengths=lengths.cuda(), save_states=True)
    out, hT, before, err, _ = ref.scan(clean(x), clean(gate), h0, lengths, "linear")
    grads = wr.delta_scan_bwd(x.cuda(), gate.cuda(), before[:, ::64].float().contiguous().cuda(), dout.cuda(),
                              dhT.cuda(), form="linear", lengths=lengths.cuda())
    torch.cuda.synchronize()
    want, gerr = ref.scan_grad(clean(x), clean(gate), h0, clean(dout), dhT, lengths, "linear")
    eb = torch.cat([torch.zeros_like(err[:, :1]), err[:, :-1]], 1)
    checks = [("out", got[0], out, torch.where(live, err, torch.zeros_like(err))), ("hT", got[1], hT, err[:, -1]), ("states", got[2], before[:, ::64], eb[:, ::64]),
              *zip(("dx", "dgate", "dh0"), grads, want, gerr)]
    # (not the runs of dips, whose gradients leave the range from other ends)
    for kind in dict.fromkeys(names):
        pick = torch.tensor([n == kind for n in names]).view(B, D)
        sel = lambda t: t.transpose(1, 2)[pick] if t.dim() == 3 else t[pick]
        for what, g, w, e in checks:
            g = g.cpu()
            if kind == "dips" and what in ("dx", "dgate", "dh0"):
                continue
            if kind in ("zeros", "still", "still_high"):
                assert torch.equal(sel(g).double(), sel(w)), f"{what} of {kind}"
            else:
                ref.within(sel(g), sel(w), sel(e) + ref.U * (sel(w).abs() + sel(e)) + LEAST, f"{what} of {kind}")
    assert not got[0].cpu()[~live.expand(B, T, D)].any()


def test_in_place_state_and_gradient():
    # the row is gone through again after other CTAs of its cluster may have ended
    names, x, gate, h0, dout, dhT = stacked(1, 1500, 32, F32, "linear", seed=2)
    state, grad = h0.cuda(), dhT.cuda()
    want = wr.delta_scan_fwd(x.cuda(), gate.cuda(), h0.cuda(), form="linear", save_states=True)
    out, hT = wr.delta_scan_fwd(x.cuda(), gate.cuda(), state, form="linear", hT=state)
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(7.0), want[0].nan_to_num(7.0))
    assert torch.equal(hT.nan_to_num(7.0), want[1].nan_to_num(7.0))


@pytest.mark.parametrize("form", ["linear", "sigmoid"])
def test_prefill_and_steps_lose_the_same_values(form):
    T = 300
    names, x, gate, h0, _, _ = stacked(1, T, 32, F32, form, seed=3)
    out, hT = wr.delta_scan_fwd(x.cuda(), gate.cuda(), h0.cuda(), form=form)
    state = h0.cuda()
    steps = torch.stack([wr.delta_scan_step(x[:, t].cuda(), gate[:, t].cuda(), state, form=form) for t in range(T)], 1)
    torch.cuda.synchronize()
    assert torch.equal(torch.isfinite(steps), torch.isfinite(out))
    assert torch.equal(torch.isnan(state), torch.isnan(hT))
