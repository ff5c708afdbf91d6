"""Workloads of three further block operators: linear attention with a decay for
each head (chunked, step, gradients), the residual addition with layer norm, and
the gated feed-forward layer, act(x Wg^T + bg) * (x Wu^T + bu).

A case names its operator in "op".  `run` computes it in plain torch operations in
32 bits, or, with `own` set, through this package's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64  # of the plain form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token for a batch of 256 sequences: 512 MiB of states, read and written once
        dict(name="decay_step_b256_h32_d128", op="decay_step", B=256, H=32, dk=128, dv=128, dtype="bf16"),
        # one decoded token for one sequence, where latency counts
        dict(name="decay_step_b1_h32_d128", op="decay_step", B=1, H=32, dk=128, dv=128, dtype="bf16"),
        # a forward over the headline batch
        dict(name="decay_fwd_b4_t8192_h32_d128", op="decay_fwd", B=4, T=8192, H=32, dk=128, dv=128,
             dtype="bf16", ragged=False),
        # one long document: few heads, so the time axis has to be split
        dict(name="decay_fwd_b1_t65536_h8_d128", op="decay_fwd", B=1, T=65536, H=8, dk=128, dv=128,
             dtype="bf16", ragged=False),
        # a right-padded batch of prompts with odd sizes, float32
        dict(name="decay_fwd_b7_t1021_h5_k64_v96", op="decay_fwd", B=7, T=1021, H=5, dk=64, dv=96,
             dtype="f32", ragged=True),
        # the gradients of a training step
        dict(name="decay_bwd_b4_t4096_h32_d128", op="decay_bwd", B=4, T=4096, H=32, dk=128, dv=128,
             dtype="bf16", ragged=False),
        # the norm of one decoded token
        dict(name="layernorm_fwd_r1_d4096", op="layernorm_fwd", rows=1, D=4096, dtype="bf16"),
        # the norm of every token of the headline batch, training forward
        dict(name="layernorm_fwd_r32768_d4096", op="layernorm_fwd", rows=32768, D=4096, dtype="bf16"),
        # its gradients, with the gradient that comes along the residual stream
        dict(name="layernorm_bwd_r32768_d2048", op="layernorm_bwd", rows=32768, D=2048, dtype="bf16"),
        # one decoded token through a feed-forward layer's first half: both weights are read once
        dict(name="glu_fwd_m1_n8192_k4096", op="glu_fwd", M=1, N=8192, K=4096, act="silu", dtype="bf16",
             save=False),
        # a whole batch through it, with what its gradients need
        dict(name="glu_fwd_m8192_n4096_k4096", op="glu_fwd", M=8192, N=4096, K=4096, act="silu",
             dtype="bf16", save=True),
        # its gradients
        dict(name="glu_bwd_m4096_n4096_k2048", op="glu_bwd", M=4096, N=4096, K=2048, act="silu",
             dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; often odd, often a multiple of 64."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    if n >= 128 and rng.random() < 0.6:
        n = n // 64 * 64
    return n


def draw(rng):
    op = rng.choice(["decay_step", "decay_fwd", "decay_fwd", "decay_fwd", "decay_bwd", "decay_bwd",
                     "layernorm_fwd", "layernorm_bwd", "glu_fwd", "glu_fwd", "glu_bwd"])
    if op.startswith("decay"):
        dk = rng.choice([128, 128, 64, rng.randrange(16, 129, 8)])
        dv = rng.choice([dk, dk, rng.randrange(16, 129, 8)])
        H = _size(rng, 1, 32)
        c = dict(op=op, H=H, dk=dk, dv=dv, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "decay_step":
            return dict(c, B=_size(rng, 1, 256))
        B = _size(rng, 1, 16)
        most = (8192 if op == "decay_fwd" else 4096) * 4 * 32 * 128
        if c["dtype"] == "f32":
            most //= 4
        T = _size(rng, 1, min(65536, most // (B * H * max(dk, dv))))
        return dict(c, B=B, T=T, ragged=rng.random() < 0.4)
    if op.startswith("layernorm"):
        D = _size(rng, 16, 8192)
        return dict(op=op, rows=_size(rng, 1, min(32768, 16384 * 4096 // D)), D=D,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    K = _size(rng, 16, 4096)
    N = _size(rng, 16, 8192)
    M = _size(rng, 1, 4096)
    c = dict(op=op, M=M, N=N, K=K, act=rng.choice(["silu", "silu", "gelu", "none"]), dtype="bf16")
    if op == "glu_fwd":
        c["save"] = rng.random() < 0.5
    return c


def _esz(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op, e = case["op"], _esz(case)
    if op.startswith("decay"):
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        heads = B * H * case.get("T", 1)
        live = 0.5 if case.get("ragged") else 1.0  # lengths are uniform: half the inputs count
        states = 8 * B * H * dk * dv + 4 * H  # one read and one written
        if op == "decay_bwd":
            return {"bytes": heads * e * (live * 2 + 1) * (dk + dv) - heads * e * dv * (1 - live) + states,
                    "flops": live * heads * 10 * dk * dv}
        return {"bytes": heads * e * (live * (2 * dk + dv) + dv) + states, "flops": live * heads * 4 * dk * dv}
    if op.startswith("layernorm"):
        r, D = case["rows"], case["D"]
        return {"bytes": r * D * 4 * e + 8 * r + 8 * D, "flops": 10 * r * D}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "glu_fwd":
        return {"bytes": e * (M * K + 2 * N * K + (3 if case["save"] else 1) * M * N) + 8 * N,
                "flops": 4 * M * N * K}
    return {"bytes": e * (2 * M * K + 4 * N * K + 3 * M * N) + 8 * N, "flops": 8 * M * N * K}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev, dt, op = torch.device("cuda"), _dtype(case), case["op"]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case)
    if op.startswith("decay"):
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        lead = (B,) if op == "decay_step" else (B, case["T"])
        # what a fused projection gives: q, k and v side by side for every token
        qkv = normal(*lead, H * (2 * dk + dv)).to(dt)
        s["q"], s["k"], s["v"] = (t.unflatten(-1, (H, -1))
                                  for t in qkv.split((H * dk, H * dk, H * dv), -1))
        # from heads that look back a few tokens to heads that look back hundreds
        s["decay"] = 1.0 - torch.exp2(-1.0 - 8.0 * torch.rand(H, generator=gen, device=dev))
        s["scale"] = dk ** -0.5
        s["h0"] = normal(B, H, dk, dv)
        if op == "decay_step":
            s["state"] = s.pop("h0")
            return s
        s["lengths"] = None
        if case["ragged"]:  # prompts from nothing to the full length
            s["lengths"] = torch.randint(0, case["T"] + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        if op == "decay_bwd":
            s["dout"] = normal(*lead, H, dv).to(dt)
            s["dhT"] = normal(B, H, dk, dv)
        return s
    if op.startswith("layernorm"):
        r, D = case["rows"], case["D"]
        loud = 1.0 + 15.0 * (torch.rand(D, generator=gen, device=dev) < 0.01)  # a few large channels
        s["weight"], s["bias"] = 1.0 + 0.1 * normal(D), 0.1 * normal(D)
        stream = normal(r, D) * 2.0 * loud + 0.5 * normal(r, 1)
        if op == "layernorm_bwd":
            s["sum"] = stream.to(dt)
            full = s["sum"].float()
            s["mean"] = full.mean(-1)
            s["rstd"] = torch.rsqrt((full - s["mean"][:, None]).square().mean(-1) + EPS)
            s["dy"], s["dsum"] = normal(r, D).to(dt), normal(r, D).to(dt)
        else:
            s["x"], s["residual"] = normal(r, D).to(dt), stream.to(dt)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["x"] = normal(M, K).to(dt)
    s["w"] = (normal(2 * N, K) / math.sqrt(K)).to(dt)  # the gate's rows, then the other projection's
    s["bias"] = 0.1 * normal(2 * N)
    if op == "glu_bwd":
        s["pre"] = (s["x"].float() @ s["w"].float().T + s["bias"]).to(dt)
        s["dout"] = normal(M, N).to(dt)
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _powers(decay, e):
    """decay^e for whole exponents, taken in 64 bits: far positions have large ones"""
    return torch.pow(decay.double().reshape(-1, *[1] * e.dim()), e.double()).float()


def _live(s):
    """[B,T], true before each row's end, and the rows' ends [B]"""
    B, T, dev = s["B"], s["T"], s["q"].device
    n = torch.full((B,), T, device=dev) if s["lengths"] is None else s["lengths"].long()
    return torch.arange(T, device=dev) < n[:, None], n


def _attend(q, k, v, decay, h0):
    """sum_{j<=t} decay^(t-j) (q_t k_j) v_j + decay^(t+1) q_t h0, over chunks of the time axis"""
    B, T, H, _ = q.shape
    n = -(-T // CHUNK)
    pad = (0, 0, 0, 0, 0, n * CHUNK - T)
    q, k, v = (torch.nn.functional.pad(t, pad).unflatten(1, (n, CHUNK)).transpose(2, 3) for t in (q, k, v))
    i = torch.arange(CHUNK, device=q.device)
    apart = i[:, None] - i
    within = torch.where(apart >= 0, _powers(decay, apart.clamp(min=0)), 0.0)
    c = torch.arange(n, device=q.device)
    back = c[:, None] - 1 - c
    between = torch.where(back >= 0, _powers(decay, CHUNK * back.clamp(min=0)), 0.0)
    own_state = (k * _powers(decay, CHUNK - 1 - i)[..., None]).transpose(-1, -2) @ v  # [B,n,H,dk,dv]
    start = torch.einsum("hcx,bxhkv->bchkv", between, own_state)
    if h0 is not None:
        start = start + _powers(decay, CHUNK * c).T[None, :, :, None, None] * h0[:, None]
    out = ((q @ k.transpose(-1, -2)) * within) @ v + (q * _powers(decay, i + 1)[..., None]) @ start
    return out.transpose(2, 3).flatten(1, 2)[:, :T]


def _gather_state(k, v, w, decay, n, h0):
    """sum_t w[b,h,t] k_t v_t^T + decay^n h0"""
    return torch.einsum("bthk,bthv->bhkv", k * w.transpose(1, 2)[..., None], v) + \
        torch.pow(decay.double(), n.double()[:, None]).float()[..., None, None] * h0


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
    if op == "decay_step":
        q, k, v = (s[n].float() for n in "qkv")
        s["state"].copy_(s["decay"][:, None, None] * s["state"] + k[..., None] * v[..., None, :])
        return {"out": (s["scale"] * (q[..., None] * s["state"]).sum(-2)).to(dt), "state": s["state"]}
    if op.startswith("decay"):
        live, n = _live(s)
        mask = live[..., None, None]
        q, k, v = (torch.where(mask, s[name].float(), 0.0) for name in "qkv")
        decay, scale, t = s["decay"], s["scale"], torch.arange(s["T"], device=live.device)
        # decay to the power of the steps that follow t in its row, 0 past its end
        left = (n[:, None] - 1 - t).clamp(min=0)
        after = torch.where(live[:, None], torch.pow(decay.double()[:, None], left.double()[:, None]).float(), 0.0)
        if op == "decay_fwd":
            out = scale * _attend(q, k, v, decay, s["h0"])
            return {"out": torch.where(mask, out, 0.0).to(dt),
                    "hT": _gather_state(k, v, after, decay, n, s["h0"])}
        do = torch.where(mask, s["dout"].float(), 0.0)
        dq = scale * _attend(do, v, k, decay, s["h0"].transpose(-1, -2))
        w = after.transpose(1, 2)[..., None]
        dv = scale * _attend(k.flip(1), q.flip(1), do.flip(1), decay, None).flip(1)
        dv = dv + torch.einsum("bthk,bhkv->bthv", k * w, s["dhT"])
        dk = scale * _attend(v.flip(1), do.flip(1), q.flip(1), decay, None).flip(1)
        dk = dk + torch.einsum("bthv,bhkv->bthk", v * w, s["dhT"])
        dh0 = _gather_state(scale * q, do, _powers(decay, t + 1)[None], decay, n, s["dhT"])
        return {"dq": torch.where(mask, dq, 0.0).to(dt), "dk": torch.where(mask, dk, 0.0).to(dt),
                "dv": torch.where(mask, dv, 0.0).to(dt), "dh0": dh0}
    if op == "layernorm_fwd":
        t = s["x"].float() + s["residual"].float()
        mean = t.mean(-1)
        rstd = torch.rsqrt((t - mean[:, None]).square().mean(-1) + EPS)
        y = (t - mean[:, None]) * rstd[:, None] * s["weight"] + s["bias"]
        return {"y": y.to(dt), "sum": t.to(dt), "mean": mean, "rstd": rstd}
    if op == "layernorm_bwd":
        that = (s["sum"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["weight"]
        dx = (g - g.mean(-1, keepdim=True) - that * (g * that).mean(-1, keepdim=True)) * s["rstd"][:, None]
        return {"dx": (dx + s["dsum"].float()).to(dt), "dweight": (dy * that).sum(0), "dbias": dy.sum(0)}
    N = s["N"]
    if op == "glu_fwd":
        pre = s["x"].float() @ s["w"].float().T + s["bias"]
        out = (_act(s["act"], pre[:, :N]) * pre[:, N:]).to(dt)
        return {"out": out, "pre": pre.to(dt)} if s["save"] else {"out": out}
    gate, up, do = s["pre"][:, :N].float(), s["pre"][:, N:].float(), s["dout"].float()
    dpre = torch.cat([do * up * _act_slope(s["act"], gate), do * _act(s["act"], gate)], -1)
    return {"dx": (dpre @ s["w"].float()).to(dt), "dw": (dpre.T @ s["x"].float()).to(dt),
            "dbias": dpre.sum(0)}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import weight_rnn_gb300 as wr

    op = s["op"]
    if op == "decay_step":
        out = wr.delta_decay_step(s["q"], s["k"], s["v"], s["decay"], s["state"], scale=s["scale"])
        return {"out": out, "state": s["state"]}
    if op == "decay_fwd":
        got = wr.delta_decay_fwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], scale=s["scale"],
                                 lengths=s["lengths"])
        return dict(zip(("out", "hT"), got))
    if op == "decay_bwd":
        got = wr.delta_decay_bwd(s["q"], s["k"], s["v"], s["decay"], s["dout"], s["h0"], s["dhT"],
                                 scale=s["scale"], lengths=s["lengths"])
        return dict(zip(("dq", "dk", "dv", "dh0"), got))
    if op == "layernorm_fwd":
        got = wr.delta_add_layernorm_fwd(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS)
        return dict(zip(("y", "sum", "mean", "rstd"), got))
    if op == "layernorm_bwd":
        got = wr.delta_add_layernorm_bwd(s["dy"], s["sum"], s["weight"], s["mean"], s["rstd"], s["dsum"])
        return dict(zip(("dx", "dweight", "dbias"), got))
    if op == "glu_fwd":
        got = wr.delta_glu_fwd(s["x"], s["w"], s["bias"], act=s["act"], save_pre=s["save"])
        return dict(zip(("out", "pre"), got)) if s["save"] else {"out": got}
    got = wr.delta_glu_bwd(s["x"], s["w"], s["dout"], s["pre"], act=s["act"])
    return dict(zip(("dx", "dw", "dbias"), got))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op.startswith("decay"):
        a = d["decay"][:, None, None]
        if op == "decay_step":
            S = a * d["state"] + torch.einsum("bhk,bhv->bhkv", d["k"], d["v"])
            return {"out": s["scale"] * torch.einsum("bhk,bhkv->bhv", d["q"], S), "state": S}
        # token by token; the last axis but one of what is looked up is the state's first
        B, T = case["B"], case["T"]
        n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
        on = torch.zeros(T, B, 1, 1, 1, dtype=torch.float64, device="cuda")
        for b in range(B):
            on[:n[b], b] = 1.0
        keep = 1.0 + on * (a - 1.0)
        for name in "qkv":
            for b in range(B):
                d[name][b, n[b]:] = 0.0

        def row(t):  # [B,H,1,d] of each token
            return t.transpose(0, 1)[:, :, :, None]

        q, k, v = row(d["q"]), row(d["k"]), row(d["v"])
        S = d["h0"]
        if op == "decay_fwd":
            out = torch.empty_like(d["v"])
            for t in range(T):
                S = torch.addcmul(k[t].transpose(-1, -2) * v[t], keep[t], S)
                out[:, t] = (q[t] @ S)[:, :, 0]
            return {"out": s["scale"] * out, "hT": S}
        for b in range(B):
            d["dout"][b, n[b]:] = 0.0
        do = s["scale"] * row(d["dout"])
        dq, dk, dv = (torch.empty_like(d[name]) for name in "qkv")
        for t in range(T):
            S = torch.addcmul(k[t].transpose(-1, -2) * v[t], keep[t], S)
            dq[:, t] = (do[t] @ S.transpose(-1, -2))[:, :, 0]
        R = d["dhT"]
        for t in range(T - 1, -1, -1):
            R = R + q[t].transpose(-1, -2) * do[t]
            dk[:, t] = (v[t] @ R.transpose(-1, -2))[:, :, 0]
            dv[:, t] = (k[t] @ R)[:, :, 0]
            R = keep[t] * R
        return {"dq": dq, "dk": dk, "dv": dv, "dh0": R}
    if op == "layernorm_fwd":
        t = d["x"] + d["residual"]
        mean = t.sum(1) / t.shape[1]
        var = t.pow(2).sum(1) / t.shape[1] - mean * mean
        rstd = 1.0 / (var + EPS).sqrt()
        y = torch.addcmul(d["bias"], d["weight"], (t - mean.unsqueeze(1)) * rstd.unsqueeze(1))
        return {"y": y, "sum": t, "mean": mean, "rstd": rstd}
    if op == "layernorm_bwd":
        r, D = d["rstd"].unsqueeze(1), case["D"]
        c = r * d["sum"] - (r * d["mean"].unsqueeze(1))
        g = torch.einsum("rd,d->rd", d["dy"], d["weight"])
        dots = torch.einsum("rd,rd->r", g, c).unsqueeze(1) / D
        return {"dx": d["dsum"] + r * g - r * (g.sum(1, keepdim=True) / D) - r * c * dots,
                "dweight": torch.einsum("rd,rd->d", d["dy"], c), "dbias": torch.einsum("rd->d", d["dy"])}
    if op == "glu_bwd":
        p = d["pre"].requires_grad_(True)
        gate, up = p.chunk(2, 1)
        (dpre,) = torch.autograd.grad(_curve(case["act"], gate) * up, p, d["dout"])
        return {"dx": torch.einsum("mn,nk->mk", dpre, d["w"]),
                "dw": torch.einsum("mn,mk->nk", dpre, d["x"]), "dbias": torch.einsum("mn->n", dpre)}
    pre = torch.einsum("mk,nk->mn", d["x"], d["w"]) + d["bias"]
    gate, up = pre.chunk(2, 1)
    out = up * _curve(case["act"], gate)
    return {"out": out, "pre": pre} if case["save"] else {"out": out}


def _curve(name, p):
    """the activations from their other forms: x sigma(x), and x sigma(2 c (x + 0.044715 x^3))"""
    if name == "silu":
        return p * torch.special.expit(p)
    if name == "gelu":
        return p * torch.special.expit(math.sqrt(8.0 / math.pi) * (p + 0.044715 * p.pow(3)))
    return p
