"""Plain 64-bit definitions of the block operators, with running bounds on what
float32 arithmetic may add, for the tests.  U is float32's rounding (half a
step), HALF a type's."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gates(gate, form):
    g = gate.double()
    if form == "linear":
        return g, torch.ones_like(g)
    return torch.special.expit(g), torch.special.expit(-g)


def _live(x, lengths):
    T = x.shape[1]
    n = torch.full((x.shape[0],), T) if lengths is None else lengths.clamp(0, T)
    return torch.arange(T)[None, :, None] < n[:, None, None]


def roundings(gate, form):
    """Relative error of one step's coefficients and sums, in units of U.  The
    sums: each step's value passes at most a map product, a map sum, the final
    recurrence and a share of the folds (8 maps a tile, 8 tiles a round): 4.
    The sigmoid adds the hardware exponential, documented as 2 + 1.173 |f| ulp
    of 2 U, and a product and a quotient of 2 ulp each on top."""
    if form == "linear":
        return torch.full_like(gate.double(), 4.0)
    return 4.0 + 2.0 * (2.0 + 1.173 * gate.double().abs().clamp(max=88.0) + 4.0)


def scan(x, gate, h0, lengths=None, form="sigmoid"):
    """out, hT, all states before each step, and bounds on the error of the
    state after each step: (out, hT, before, err_after, abs_after)."""
    B, T, D = x.shape
    a, u = gates(gate, form)
    live = _live(x, lengths)
    k = roundings(gate, form) * U
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    big, err = h.abs(), torch.zeros_like(h)
    out, before, errs, bigs = ([] for _ in range(4))
    for t in range(T):
        on, at, bt = live[:, t], a[:, t], u[:, t] * x[:, t].double()
        before.append(h)
        keep = at != 0  # a reset drops the state, whatever it holds
        h_new = torch.where(keep, at * h, 0.0) + bt
        big_new = torch.where(keep, at.abs() * big, 0.0) + bt.abs()
        err_new = torch.where(keep, at.abs() * err, 0.0) + k[:, t] * big_new
        h, big, err = (torch.where(on, n, o) for n, o in ((h_new, h), (big_new, big), (err_new, err)))
        out.append(torch.where(on, h, 0.0))
        errs.append(err)
        bigs.append(big)
    stack = lambda v: torch.stack(v, 1) if v else torch.zeros(B, 0, D, dtype=torch.float64)
    return stack(out), h, stack(before), stack(errs), stack(bigs)


def scan_grad(x, gate, h0, dout, dhT, lengths=None, form="sigmoid"):
    """(dx, dgate, dh0) and their bounds, without the final rounding."""
    B, T, D = x.shape
    a, u = gates(gate, form)
    live = _live(x, lengths)
    k = roundings(gate, form) * U
    _, _, before, err_after, big_after = scan(x, gate, h0, lengths, form)
    h0d = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    err_b = torch.cat([torch.zeros(B, 1, D, dtype=torch.float64), err_after[:, :-1]], 1)
    big_b = torch.cat([h0d.abs()[:, None], big_after[:, :-1]], 1)
    c = torch.zeros(B, D, dtype=torch.float64) if dhT is None else dhT.double()
    big, err = c.abs(), torch.zeros_like(c)
    dx, dg, ex, eg = (torch.zeros(B, T, D, dtype=torch.float64) for _ in range(4))
    for t in range(T - 1, -1, -1):
        on, at, ut = live[:, t], a[:, t], u[:, t]
        do = dout[:, t].double()
        dh, bigh = do + c, do.abs() + big
        eh = err + U * bigh
        xv = x[:, t].double()
        if form == "linear":
            g, eg_t = dh * before[:, t], eh * big_b[:, t] + bigh * err_b[:, t]
            eg_t = eg_t + 2 * k[:, t] * bigh * big_b[:, t]
        else:
            g = dh * at * ut * (before[:, t] - xv)
            s = big_b[:, t] + xv.abs()
            eg_t = at * ut * (eh * s + bigh * err_b[:, t] + 3 * k[:, t] * bigh * s)
        zero = torch.zeros_like(dh)
        dx[:, t], dg[:, t] = torch.where(on, ut * dh, zero), torch.where(on, g, zero)
        ex[:, t] = torch.where(on, ut * (eh + k[:, t] * bigh), zero)
        eg[:, t] = torch.where(on, eg_t, zero)
        keep = at != 0
        cn = torch.where(keep, at * dh, zero)
        bn = torch.where(keep, at.abs() * bigh, zero)
        en = torch.where(keep, at.abs() * eh, zero) + k[:, t] * bn
        c, big, err = (torch.where(on, n, o) for n, o in ((cn, c), (bn, big), (en, err)))
    return (dx, dg, c), (ex, eg, err)


def norm(x, residual, weight, eps):
    t = x.double() + (0.0 if residual is None else residual.double())
    rstd = (t.square().mean(-1) + eps).rsqrt()
    return t, rstd, t * rstd[..., None] * weight.double()


def norm_grad(dy, total, weight, rstd, dsum):
    """(dx, dweight), and the sums of magnitudes that bound their roundings"""
    that = total.double() * rstd.double()[..., None]
    g = dy.double() * weight.double()
    ds = torch.zeros_like(g) if dsum is None else dsum.double()
    r = rstd.double()[..., None]
    dx = r * (g - that * (g * that).mean(-1, keepdim=True)) + ds
    big = r * (g.abs() + that.abs() * (g * that).abs().mean(-1, keepdim=True)) + ds.abs()
    flat = (dy.double() * that).reshape(-1, dy.shape[-1])
    return (dx, flat.sum(0)), (big, flat.abs().sum(0))


def act(name, p):
    if name == "silu":
        return p * torch.special.expit(p)
    if name == "gelu":
        return p * torch.special.expit((8.0 / torch.pi) ** 0.5 * (p + 0.044715 * p ** 3))
    return p


def within(got, ref, err, what):
    """Element by element: |got - ref| <= err."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), f"{what}: finite elsewhere"
    off = (got - ref).abs() - err
    off = torch.where(torch.isfinite(ref), off, torch.zeros_like(off))
    if off.numel():
        worst = off.max().item()
        at = off.argmax().item()
        assert worst <= 0, (f"{what}: off by {(got - ref).abs().flatten()[at]:.3e} at {at}, "
                            f"allowed {torch.as_tensor(err).expand_as(ref).flatten()[at]:.3e}")
