"""Workloads of the block operators: the gated linear recurrence (scan), the residual
addition with RMS norm, and the linear layer with its epilogue, each forward and
backward and in its form for single tokens.

A case names its operator in "op".  `run` computes it in plain torch operations in
32 bits, or, with `own` set, through this package's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 64  # steps between two saved states of the recurrence
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token for a batch of 256 sequences: the state is read and written once
        dict(name="scan_step_b256_d4096", op="scan_step", B=256, D=4096, form="sigmoid", dtype="bf16"),
        # a training forward over the headline batch, states kept for the backward pass
        dict(name="scan_fwd_b4_t8192_d4096", op="scan_fwd", B=4, T=8192, D=4096, form="sigmoid",
             dtype="bf16", ragged=False, save=True),
        # one long document: few channels, so the time axis has to be split
        dict(name="scan_fwd_b1_t65536_d2048", op="scan_fwd", B=1, T=65536, D=2048, form="linear",
             dtype="bf16", ragged=False, save=False),
        # a right-padded batch of prompts with odd sizes, float32
        dict(name="scan_fwd_b7_t1021_d1001", op="scan_fwd", B=7, T=1021, D=1001, form="sigmoid",
             dtype="f32", ragged=True, save=False),
        # the gradients of a training step
        dict(name="scan_bwd_b8_t4096_d2048", op="scan_bwd", B=8, T=4096, D=2048, form="sigmoid",
             dtype="bf16", ragged=False),
        # decoding one token: the norm before an 8-bit projection, where latency counts
        dict(name="norm_quant_r1_d4096", op="norm_quant", rows=1, D=4096, dtype="bf16"),
        # the norm of every token of the headline batch, training forward
        dict(name="norm_fwd_r32768_d4096", op="norm_fwd", rows=32768, D=4096, dtype="bf16"),
        # its gradients, with the gradient that comes along the residual stream
        dict(name="norm_bwd_r32768_d2048", op="norm_bwd", rows=32768, D=2048, dtype="bf16"),
        # decoding one token through a projection: the weight is read once
        dict(name="linear_fwd_m1_n8192_k4096", op="linear_fwd", M=1, N=8192, K=4096, act="silu",
             dtype="bf16", save=False),
        # a projection over a whole batch with everything in its epilogue
        dict(name="linear_fwd_m8192_n4096_k4096", op="linear_fwd", M=8192, N=4096, K=4096,
             act="silu", dtype="bf16", save=True),
        # a prefill of odd length through an 8-bit projection
        dict(name="linear_quant_m4099_n4096_k4096", op="linear_quant", M=4099, N=4096, K=4096,
             act="gelu", dtype="bf16"),
        # the gradients of a projection
        dict(name="linear_bwd_m4096_n4096_k2048", op="linear_bwd", M=4096, N=4096, K=2048,
             act="silu", dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; often odd, often a multiple of 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    if n >= 128 and rng.random() < 0.6:
        n = n // 64 * 64
    return n


def draw(rng):
    op = rng.choice(["scan_step", "scan_fwd", "scan_fwd", "scan_bwd", "norm_fwd", "norm_quant",
                     "norm_bwd", "linear_fwd", "linear_fwd", "linear_quant", "linear_bwd"])
    if op == "scan_step":
        return dict(op=op, B=_size(rng, 1, 256), D=_size(rng, 16, 4096),
                    form=rng.choice(["sigmoid", "linear"]), dtype=rng.choice(["bf16", "f32"]))
    if op in ("scan_fwd", "scan_bwd"):
        most = 8 * 4096 * 2048
        D = _size(rng, 16, 4096)
        B = _size(rng, 1, 16)
        T = _size(rng, 1, min(65536, most // (B * D)))
        c = dict(op=op, B=B, T=T, D=D, form=rng.choice(["sigmoid", "linear"]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.4)
        if op == "scan_fwd":
            c["save"] = rng.random() < 0.5
        return c
    if op.startswith("norm"):
        D = _size(rng, 16, 8192)
        return dict(op=op, rows=_size(rng, 1, min(32768, 16384 * 4096 // D)), D=D,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    K = _size(rng, 16, 4096)
    N = _size(rng, 16, 8192)
    M = _size(rng, 1, 4096)
    c = dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "silu", "gelu"]), dtype="bf16")
    if op == "linear_fwd":
        c["save"] = rng.random() < 0.5
    return c


def _esz(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op, e = case["op"], _esz(case)
    if op.startswith("scan"):
        B, D, T = case["B"], case["D"], case.get("T", 1)
        n, g = B * T * D, e if case["form"] == "sigmoid" else 4
        if op == "scan_step":
            return {"bytes": n * (2 * e + g + 8), "flops": 10 * n}
        states = 4 * B * D * (-(-T // BLOCK))
        live = 0.5 if case["ragged"] else 1.0  # lengths are uniform: half the inputs count
        if op == "scan_fwd":
            return {"bytes": n * (live * (e + g) + e) + 8 * B * D + (states if case["save"] else 0),
                    "flops": 10 * n}
        return {"bytes": n * (live * (2 * e + g) + e + g) + states + 8 * B * D, "flops": 20 * n}
    if op.startswith("norm"):
        r, D = case["rows"], case["D"]
        per = {"norm_fwd": 4 * e, "norm_quant": 3 * e + 1, "norm_bwd": 4 * e}[op]
        return {"bytes": r * D * per + 4 * r + 4 * D, "flops": 8 * r * D}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_fwd":
        return {"bytes": e * (M * K + N * K + (3 if case["save"] else 2) * M * N) + 4 * N,
                "flops": 2 * M * N * K}
    if op == "linear_quant":
        return {"bytes": M * K + N * K + 2 * e * M * N + 4 * (M + 2 * N), "flops": 2 * M * N * K}
    return {"bytes": e * (2 * M * K + 2 * N * K + 2 * M * N) + 4 * N, "flops": 4 * M * N * K}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev, dt, op = torch.device("cuda"), _dtype(case), case["op"]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case)
    if op.startswith("scan"):
        B, D = case["B"], case["D"]
        lead = (B, D) if op == "scan_step" else (B, case["T"], D)
        s["x"] = normal(*lead).to(dt)
        if case["form"] == "sigmoid":
            s["gate"] = (normal(*lead) * 1.5 + 2.5).to(dt)
        else:  # decays near one, and a reset here and there where a document ends
            g = torch.exp(-0.1 * torch.log1p(torch.exp(normal(*lead))))
            cut = torch.rand(*lead[:-1], 1, generator=gen, device=dev) < 1.0 / 512
            s["gate"] = g.masked_fill(cut, 0.0)
        s["h0"] = normal(B, D)
        if op == "scan_step":
            s["state"] = s.pop("h0")
            return s
        s["lengths"] = None
        if case["ragged"]:  # prompts from nothing to the full length
            s["lengths"] = torch.randint(0, case["T"] + 1, (B,), generator=gen, device=dev,
                                         dtype=torch.int32)
        if op == "scan_bwd":
            s["dout"] = normal(*lead).to(dt)
            s["dhT"] = normal(B, D)
            h = _states(s)
            before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
            s["states"] = before[:, ::BLOCK].contiguous()
        return s
    if op.startswith("norm"):
        r, D = case["rows"], case["D"]
        loud = 1.0 + 15.0 * (torch.rand(D, generator=gen, device=dev) < 0.01)  # a few large channels
        s["weight"] = (1.0 + 0.1 * normal(D)).float()
        if op == "norm_bwd":
            full = normal(r, D) * 2.0 * loud
            s["sum"] = full.to(dt)
            s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(-1) + EPS)
            s["dy"], s["dsum"] = normal(r, D).to(dt), normal(r, D).to(dt)
        else:
            s["x"] = normal(r, D).to(dt)
            s["residual"] = (normal(r, D) * 2.0 * loud).to(dt)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    x, w = normal(M, K), normal(N, K) / math.sqrt(K)
    s["bias"] = 0.1 * normal(N)
    if op == "linear_quant":
        for n, t in (("x", x), ("w", w)):
            scale = t.abs().amax(-1) / E4M3_MAX
            s[n] = (t / scale[:, None]).to(torch.float8_e4m3fn)
            s[n + "_scale"] = scale
    else:
        s["x"], s["w"] = x.to(dt), w.to(dt)
    if op == "linear_bwd":
        s["pre"] = (s["x"].float() @ s["w"].float().T + s["bias"]).to(dt)
        s["dout"] = normal(M, N).to(dt)
    else:
        s["residual"] = normal(M, N).to(dt)
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0, along dim 1, by doubling the span that each entry covers."""
    d, T = 1, a.shape[1]
    while d < T:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _gates(s, axis=True):
    """decay a, its complement (1 - a, or 1 in the linear form), input x, and which steps count"""
    x, g = s["x"].float(), s["gate"].float()
    if s["form"] == "sigmoid":
        a, u = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    else:
        a, u = g, torch.ones_like(g)
    if not axis or s["lengths"] is None:
        return a, u, x, None
    live = (torch.arange(x.shape[1], device=x.device)[None] < s["lengths"][:, None])[..., None]
    return torch.where(live, a, 1.0), torch.where(live, u, 0.0), x, live


def _states(s):
    """every h_t, with steps past a row's length leaving it alone"""
    a, u, x, _ = _gates(s)
    b = u * x
    b[:, 0] += a[:, 0] * s["h0"]
    return _scan(a, b)


def _act(name, p):
    if name == "silu":
        return p / (1.0 + torch.exp(-p))
    if name == "gelu":  # the tanh form
        return 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p * p * p)))
    return p


def _act_slope(name, p):
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-p))
        return sg * (1.0 + p * (1.0 - sg))
    if name == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (p + 0.044715 * p * p * p))
        return 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * p * p)
    return torch.ones_like(p)


def _plain(s):
    op, dt = s["op"], _dtype(s)
    if op == "scan_step":
        a, u, x, _ = _gates(s, axis=False)
        s["state"].copy_(a * s["state"] + u * x)
        return {"out": s["state"].to(dt), "state": s["state"]}
    if op == "scan_fwd":
        h = _states(s)
        got = {"hT": h[:, -1].contiguous()}
        if s["save"]:
            got["states"] = torch.cat([s["h0"][:, None], h[:, :-1]], 1)[:, ::BLOCK].contiguous()
        live = _gates(s)[3] if s["ragged"] else None
        got["out"] = (h if live is None else torch.where(live, h, 0.0)).to(dt)
        return got
    if op == "scan_bwd":
        a, u, x, live = _gates(s)
        h = _states(s)
        before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
        do = s["dout"].float() if live is None else torch.where(live, s["dout"].float(), 0.0)
        do = do.clone()
        do[:, -1] += s["dhT"]
        after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # the decay that follows each step
        dh = _scan(after.flip(1), do.flip(1)).flip(1)
        if s["form"] == "sigmoid":
            dx, dg = u * dh, dh * a * u * (before - x)
        else:
            dx, dg = u * dh, dh * before
        if live is not None:
            dx, dg = torch.where(live, dx, 0.0), torch.where(live, dg, 0.0)
        return {"dx": dx.to(dt), "dgate": dg.to(s["gate"].dtype), "dh0": a[:, 0] * dh[:, 0]}
    if op in ("norm_fwd", "norm_quant"):
        t = s["x"].float() + s["residual"].float()
        rstd = torch.rsqrt(t.square().mean(-1) + EPS)
        y = t * rstd[:, None] * s["weight"]
        if op == "norm_fwd":
            return {"y": y.to(dt), "sum": t.to(dt), "rstd": rstd}
        top = y.abs().amax(-1)
        scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
        return {"y": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale, "sum": t.to(dt)}
    if op == "norm_bwd":
        that = s["sum"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        wdy = dy * s["weight"]
        dt_ = (wdy - that * (wdy * that).mean(-1, keepdim=True)) * s["rstd"][:, None]
        return {"dx": (dt_ + s["dsum"].float()).to(dt), "dweight": (dy * that).sum(0)}
    if op == "linear_fwd":
        pre = s["x"].float() @ s["w"].float().T + s["bias"]
        out = (_act(s["act"], pre) + s["residual"].float()).to(dt)
        return {"out": out, "pre": pre.to(dt)} if s["save"] else {"out": out}
    if op == "linear_quant":
        pre = (s["x"].float() * s["x_scale"][:, None]) @ (s["w"].float() * s["w_scale"][:, None]).T
        return {"out": (_act(s["act"], pre + s["bias"]) + s["residual"].float()).to(dt)}
    dpre = s["dout"].float() * _act_slope(s["act"], s["pre"].float())
    return {"dx": (dpre @ s["w"].float()).to(dt), "dw": (dpre.T @ s["x"].float()).to(dt),
            "dbias": dpre.sum(0)}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import weight_rnn_gb300 as wr

    op = s["op"]
    if op == "scan_step":
        out = wr.delta_scan_step(s["x"], s["gate"], s["state"], form=s["form"])
        return {"out": out, "state": s["state"]}
    if op == "scan_fwd":
        got = wr.delta_scan_fwd(s["x"], s["gate"], s["h0"], form=s["form"], lengths=s["lengths"],
                                save_states=s["save"])
        return dict(zip(("out", "hT", "states"), got))
    if op == "scan_bwd":
        got = wr.delta_scan_bwd(s["x"], s["gate"], s["states"], s["dout"], s["dhT"],
                                form=s["form"], lengths=s["lengths"])
        return dict(zip(("dx", "dgate", "dh0"), got))
    if op == "norm_fwd":
        got = wr.delta_add_rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=EPS)
        return dict(zip(("y", "sum", "rstd"), got))
    if op == "norm_quant":
        got = wr.delta_add_rmsnorm_quant(s["x"], s["weight"], s["residual"], eps=EPS)
        return dict(zip(("y", "scale", "sum"), got))
    if op == "norm_bwd":
        got = wr.delta_add_rmsnorm_bwd(s["dy"], s["sum"], s["weight"], s["rstd"], s["dsum"])
        return dict(zip(("dx", "dweight"), got))
    if op == "linear_fwd":
        got = wr.delta_linear_fwd(s["x"], s["w"], s["bias"], s["residual"], act=s["act"],
                                  save_pre=s["save"])
        return dict(zip(("out", "pre"), got)) if s["save"] else {"out": got}
    if op == "linear_quant":
        return {"out": wr.delta_linear_quant(s["x"], s["x_scale"], s["w"], s["w_scale"], s["bias"],
                                             s["residual"], act=s["act"])}
    got = wr.delta_linear_bwd(s["x"], s["w"], s["dout"], s["pre"], act=s["act"])
    return dict(zip(("dx", "dw", "dbias"), got))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    # (an 8-bit value is widened by way of 32 bits, which hold it exactly)
    d = {k: (v.float() if v.dtype == torch.float8_e4m3fn else v).double()
         for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op.startswith("scan"):
        a, x = d["gate"], d["x"]
        keep = 1.0
        if case["form"] == "sigmoid":
            keep = torch.special.expit(-a)
            a = torch.special.expit(a)
        u = keep * x
        if op == "scan_step":
            h = torch.addcmul(u, a, d["state"])
            return {"out": h, "state": h}
        B, T, D = x.shape
        n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
        for b in range(B):
            a[b, n[b]:], u[b, n[b]:] = 1.0, 0.0
        h = torch.empty(B, T + 1, D, dtype=torch.float64, device=x.device)
        h[:, 0] = d["h0"]
        for t in range(T):
            torch.addcmul(u[:, t], a[:, t], h[:, t], out=h[:, t + 1])
        if op == "scan_fwd":
            got = {"hT": h[:, T].clone()}
            if case["save"]:
                got["states"] = h[:, 0:T:BLOCK].clone()
            out = h[:, 1:]
            for b in range(B):
                out[b, n[b]:] = 0.0
            return {**got, "out": out}
        do = d["dout"]
        for b in range(B):
            do[b, n[b]:] = 0.0
        dh = torch.empty_like(do)
        c = d["dhT"]
        for t in range(T - 1, -1, -1):
            dh[:, t] = do[:, t] + c
            c = a[:, t] * dh[:, t]
        dx = keep * dh
        dg = dh * h[:, :-1] if case["form"] == "linear" else dh * a * keep * (h[:, :-1] - x)
        for b in range(B):
            dx[b, n[b]:], dg[b, n[b]:] = 0.0, 0.0
        return {"dx": dx, "dgate": dg, "dh0": c}
    if op in ("norm_fwd", "norm_quant"):
        t = d["x"] + d["residual"]
        rms = (t.pow(2).sum(1) / t.shape[1] + EPS).sqrt()
        y = d["weight"] * t / rms.unsqueeze(1)
        if op == "norm_fwd":
            return {"y": y, "sum": t, "rstd": 1.0 / rms}
        scale = y.abs().max(1).values / E4M3_MAX
        scale = scale.masked_fill(scale == 0, 1.0)
        return {"y": y / scale.unsqueeze(1), "scale": scale, "sum": t}
    if op == "norm_bwd":
        r = d["rstd"].unsqueeze(1)
        t, g = d["sum"], d["dy"] * d["weight"]
        inner = torch.einsum("rd,rd->r", g, t).unsqueeze(1) / t.shape[1]
        return {"dx": r * g - r.pow(3) * inner * t + d["dsum"],
                "dweight": torch.einsum("rd,rd->d", d["dy"], r * t)}
    if op == "linear_bwd":
        p = d["pre"].requires_grad_(True)
        (dpre,) = torch.autograd.grad(_curve(case["act"], p), p, d["dout"])
        return {"dx": torch.einsum("mn,nk->mk", dpre, d["w"]),
                "dw": torch.einsum("mn,mk->nk", dpre, d["x"]), "dbias": dpre.sum(0)}
    pre = torch.einsum("mk,nk->mn", d["x"], d["w"])
    if op == "linear_quant":
        pre = pre * torch.outer(d["x_scale"], d["w_scale"])
    pre = pre + d["bias"]
    out = _curve(case["act"], pre) + d["residual"]
    return {"out": out, "pre": pre} if case.get("save") else {"out": out}


def _curve(name, p):
    """the activations from their other forms: x sigma(x), and x sigma(2 c (x + 0.044715 x^3))"""
    if name == "silu":
        return p * torch.special.expit(p)
    if name == "gelu":
        return p * torch.special.expit(math.sqrt(8.0 / math.pi) * (p + 0.044715 * p.pow(3)))
    return p
