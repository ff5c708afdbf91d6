"""Operators around the token mixers in a block: the gated linear recurrence
(``delta_scan_*``), linear attention with a decay for each head
(``delta_decay_*``), the residual addition with RMS norm
(``delta_add_rmsnorm_*``) or layer norm (``delta_add_layernorm_*``), the linear layer with its epilogue
(``delta_linear_*``) and the gated feed-forward layer (``delta_glu_*``).

Bindings over the C ABI of ``libdelta.so`` with the ABI's names: argument
checks, output allocation, the current CUDA stream, statuses as exceptions.
The common case (plain CUDA tensors that fit, outputs to be allocated, the
current stream) is taken by the compiled module ``_fast``; what that does not
take is checked and called here, with the same results.
With ``stream=`` the outputs are allocated for that stream; inputs made on
another stream are the caller's to order and to keep, as with any kernel.
None of the calls takes part in autograd, like the mixers': outputs carry no
gradient function whatever their inputs ask for, and the gradients are calls of
their own.  Tensors may be on any device; their own is made current for a call.
"""
from __future__ import annotations

import ctypes

import torch

DELTA_SCAN_LINEAR = 0
DELTA_SCAN_SIGMOID = 1
_SCAN_FORMS = {"linear": DELTA_SCAN_LINEAR, "sigmoid": DELTA_SCAN_SIGMOID}
SCAN_BLOCK = 64  # steps between two saved states
DELTA_ACT_NONE = 0
DELTA_ACT_SILU = 1
DELTA_ACT_GELU = 2
_ACTS = {"none": DELTA_ACT_NONE, "silu": DELTA_ACT_SILU, "gelu": DELTA_ACT_GELU}
_CODES = {torch.float32: 0, torch.bfloat16: 1}
E4M3 = torch.float8_e4m3fn

SYMBOLS = ("delta_scan_fwd", "delta_scan_step", "delta_scan_bwd", "delta_decay_fwd",
           "delta_decay_step", "delta_decay_bwd", "delta_add_rmsnorm_fwd",
           "delta_add_rmsnorm_quant", "delta_add_rmsnorm_bwd", "delta_add_layernorm_fwd",
           "delta_add_layernorm_bwd", "delta_linear_fwd",
           "delta_linear_quant", "delta_linear_bwd", "delta_glu_fwd", "delta_glu_bwd")


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    p, i, n, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    for name, args in (
            ("delta_scan_fwd", [p] * 7 + [i] * 3 + [n] * 4 + [i] * 2 + [p]),
            ("delta_scan_step", [p] * 4 + [i] * 2 + [n] * 2 + [i] * 2 + [p]),
            ("delta_scan_bwd", [p] * 9 + [i] * 3 + [n] * 4 + [i] * 2 + [p]),
            ("delta_decay_fwd", [p] * 8 + [i] * 5 + [p, f, i, p]),
            ("delta_decay_step", [p] * 6 + [i] * 4 + [p, f, i, p]),
            ("delta_decay_bwd", [p] * 12 + [i] * 5 + [p, f, i, p]),
            ("delta_add_rmsnorm_fwd", [p] * 6 + [n, i, n, n, f, i, i, p]),
            ("delta_add_rmsnorm_quant", [p] * 6 + [n, i, n, n, f, i, i, p]),
            ("delta_add_rmsnorm_bwd", [p] * 7 + [n, i, i, i, p]),
            ("delta_add_layernorm_fwd", [p] * 8 + [n, i, n, n, f, i, i, i, p]),
            ("delta_add_layernorm_bwd", [p] * 9 + [n, i, i, i, p]),
            ("delta_linear_fwd", [p] * 6 + [i] * 3 + [n] * 3 + [i] * 3 + [p]),
            ("delta_linear_quant", [p] * 7 + [i] * 3 + [n] * 3 + [i] * 2 + [p]),
            ("delta_linear_bwd", [p] * 7 + [i] * 3 + [n] * 2 + [i] * 2 + [p]),
            ("delta_glu_fwd", [p] * 5 + [i] * 3 + [n] * 2 + [i] * 3 + [p]),
            ("delta_glu_bwd", [p] * 7 + [i] * 3 + [n] * 2 + [i] * 2 + [p])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = i, args


def _lib():
    from . import load_library
    global _lib
    lib = load_library()
    _lib = lambda: lib  # noqa: E731  (the library stays open for the process)
    return lib


class _Nothing:
    """Stands for ``_fast`` where it was not built."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


_fast = None


def _open_fast():
    global _fast
    _lib()
    try:
        from . import _fast as module
    except ImportError:
        module = _Nothing()
    _fast = module
    return module


def _checked(r):
    """The compiled module's answer: outputs, or a status to raise."""
    if type(r) is int:
        _raise(r)
    return r


def _raise(st):
    from . import DeltaError, delta_last_error
    raise DeltaError(st, delta_last_error())


def _refuse(t, name, shape, dtype, device, strided):
    """Say what is wrong with a tensor that did not pass."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"the last axis of {name} must be contiguous" if strided
                     else f"{name} must be contiguous")


def _tensor(t, name, shape, dtype, device, strided=False):
    """Check one tensor and give its address; with ``strided`` any non-negative
    strides with contiguous rows are taken, else it has to be contiguous."""
    try:
        if t.shape == shape and t.dtype is dtype and t.device == device and (
                t.is_contiguous() or strided and (t.shape[-1] <= 1 or t.stride(-1) == 1)):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, device, strided)


def _optional(t, name, shape, dtype, device):
    return None if t is None else _tensor(t, name, shape, dtype, device)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(dev, fn):
    """A call of the library with the tensors' device current: it launches,
    allocates scratch and asks for the number of SMs on the current one, and the
    default stream's handle is the same on every device."""
    if dev.index == _current_device():
        return fn

    def call(*args):
        with torch.cuda.device(dev):
            return fn(*args)
    return call


_MOST = (1 << 31) - 1


def _within_int(what, sizes):
    """The ABI's sizes are C ints, which ctypes would cut without a word."""
    if sizes and max(sizes) > _MOST:
        raise ValueError(f"{what} has a size of {max(sizes)}, the most is 2^31 - 1")


def _begin(x, name, dims, what="x"):
    """dtype code and device of the operator's leading tensor, whose `dims` axes
    (or, with 0, whose last one) are sizes of the call"""
    try:
        dev, dt = x.device, x.dtype
    except AttributeError:
        raise TypeError(f"{what} must be a torch.Tensor") from None
    if dev.type != "cuda":
        raise ValueError(f"{name} needs CUDA tensors")
    if dims and x.dim() != dims:
        raise ValueError(f"{what} must have {dims} axes, got shape {tuple(x.shape)}")
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float32, got {dt}")
    _within_int(what, x.shape if dims else x.shape[-1:])
    return code, dev


def _raw_stream(dev, stream):
    """The stream's handle.  The current one is asked for by device index,
    which takes a twentieth of what making a Stream object does (2 us, as much
    as the launch)."""
    return _current(dev.index) if stream is None else stream.cuda_stream


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_current = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _empty(shape, dtype, dev, stream):
    """An output, allocated for the stream of the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _output(t, name, shape, dtype, dev, stream):
    if t is None:
        return _empty(shape, dtype, dev, stream)
    _tensor(t, name, shape, dtype, dev)
    return t


def _scan_form(form, dt):
    code = _SCAN_FORMS.get(form)
    if code is None:
        raise ValueError(f"form must be one of {sorted(_SCAN_FORMS)}, got {form!r}")
    return code, (torch.float32 if code == DELTA_SCAN_LINEAR else dt)


def delta_scan_fwd(x, gate, h0=None, *, form="sigmoid", lengths=None, save_states=False,
                   out=None, hT=None, stream=None):
    """Gated linear recurrence ``h_t = a_t h_{t-1} + u_t x_t`` per channel.

    x [B,T,D] bfloat16 or float32.  ``form="sigmoid"``: gate [B,T,D] in x's
    type holds logits, a = sigmoid(gate), u = 1 - a.  ``form="linear"``: gate
    [B,T,D] float32 is a itself, u = 1, and a = 0 drops the state whatever it
    holds.  x and gate may be slices (contiguous last axis).  h0 [B,D] float32
    or None; lengths [B] int32: later steps are not read, leave the state
    alone and have out = 0.  Returns ``(out [B,T,D], hT [B,D] float32)``, and
    with ``save_states`` the states [B, ceil(T/64), D] that ``delta_scan_bwd``
    takes.  ``hT`` may be ``h0`` to update the state in place.
    """
    if stream is None and out is None and hT is None:
        r = (_fast or _open_fast()).scan_fwd(x, gate, h0, lengths, save_states,
                                             _SCAN_FORMS.get(form, -1))
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(x, "delta_scan_fwd", 3)
    B, T, D = x.shape
    fcode, gdt = _scan_form(form, x.dtype)
    px = _tensor(x, "x", x.shape, x.dtype, dev, True)
    pg = _tensor(gate, "gate", x.shape, gdt, dev, True)
    ph = _optional(h0, "h0", (B, D), torch.float32, dev)
    pl = _optional(lengths, "lengths", (B,), torch.int32, dev)
    out = _output(out, "out", (B, T, D), x.dtype, dev, stream)
    hT = _output(hT, "hT", (B, D), torch.float32, dev, stream)
    states = _empty((B, -(-T // SCAN_BLOCK), D), torch.float32, dev, stream) if save_states else None
    st = _on(dev, _lib().delta_scan_fwd)(px, pg, ph, pl, out.data_ptr(), hT.data_ptr(),
        None if states is None else states.data_ptr(), B, T, D, x.stride(0), x.stride(1),
        gate.stride(0), gate.stride(1), code, fcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return (out, hT, states) if save_states else (out, hT)


def delta_scan_step(x, gate, state, *, form="sigmoid", out=None, stream=None):
    """One step of the recurrence: x, gate [B,D] (rows may be strided), state
    [B,D] float32 updated in place.  Returns out [B,D] in x's type."""
    if stream is None and out is None:
        r = (_fast or _open_fast()).scan_step(x, gate, state, _SCAN_FORMS.get(form, -1))
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(x, "delta_scan_step", 2)
    B, D = x.shape
    fcode, gdt = _scan_form(form, x.dtype)
    px = _tensor(x, "x", x.shape, x.dtype, dev, True)
    pg = _tensor(gate, "gate", x.shape, gdt, dev, True)
    ps = _tensor(state, "state", x.shape, torch.float32, dev)
    out = _output(out, "out", x.shape, x.dtype, dev, stream)
    st = _on(dev, _lib().delta_scan_step)(px, pg, ps, out.data_ptr(), B, D, x.stride(0),
        gate.stride(0), code, fcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return out


def delta_scan_bwd(x, gate, states, dout, dhT=None, *, form="sigmoid", lengths=None, stream=None):
    """Gradients of ``delta_scan_fwd``: x, gate, lengths as there, the states
    it saved, dout [B,T,D] contiguous in x's type, dhT [B,D] float32 or None.
    Returns ``(dx, dgate, dh0)``: dx in x's type, dgate in gate's, dh0 float32.
    """
    if stream is None:
        r = (_fast or _open_fast()).scan_bwd(x, gate, states, dout, dhT, lengths,
                                             _SCAN_FORMS.get(form, -1))
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(x, "delta_scan_bwd", 3)
    B, T, D = x.shape
    fcode, gdt = _scan_form(form, x.dtype)
    px = _tensor(x, "x", x.shape, x.dtype, dev, True)
    pg = _tensor(gate, "gate", x.shape, gdt, dev, True)
    ps = _tensor(states, "states", (B, -(-T // SCAN_BLOCK), D), torch.float32, dev)
    po = _tensor(dout, "dout", x.shape, x.dtype, dev)
    pt = _optional(dhT, "dhT", (B, D), torch.float32, dev)
    pl = _optional(lengths, "lengths", (B,), torch.int32, dev)
    dx, dgate = _empty(x.shape, x.dtype, dev, stream), _empty(x.shape, gdt, dev, stream)
    dh0 = _empty((B, D), torch.float32, dev, stream)
    st = _on(dev, _lib().delta_scan_bwd)(px, pg, ps, pl, po, pt, dx.data_ptr(), dgate.data_ptr(),
        dh0.data_ptr(), B, T, D, x.stride(0), x.stride(1), gate.stride(0), gate.stride(1), code,
        fcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return dx, dgate, dh0


def _decay_begin(q, k, v, decay, dims, name):
    """shared checks: types, sizes, pointers, and the strides of all axes but the last"""
    code, dev = _begin(q, name, dims, "q")
    if not isinstance(v, torch.Tensor) or v.dim() != dims:
        raise ValueError(f"v must have {dims} axes")
    _within_int("v", v.shape)
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    pq = _tensor(q, "q", q.shape, q.dtype, dev, True)
    pk = _tensor(k, "k", q.shape, q.dtype, dev, True)
    pv = _tensor(v, "v", q.shape[:-1] + (dv,), q.dtype, dev, True)
    pd = _tensor(decay, "decay", (H,), torch.float32, dev)
    strides = [n for t in (q, k, v) for n in t.stride()[:-1]]
    return code, dev, H, dk, dv, pq, pk, pv, pd, (ctypes.c_int64 * len(strides))(*strides)


def delta_decay_fwd(q, k, v, decay, h0=None, *, scale=1.0, lengths=None, out=None, hT=None, stream=None):
    """Linear attention with a decay for each head: ``S_t = decay_h S_{t-1} + k_t v_t^T``,
    ``out_t = scale S_t^T q_t``.

    q, k [B,T,H,dk] and v [B,T,H,dv] bfloat16 or float32 (contiguous last axis, dk and
    dv up to 256), decay [H] float32 in [0, 1], h0 [B,H,dk,dv] float32 or None;
    lengths [B] int32: later tokens do not count, leave the state alone and have
    out = 0.  Returns ``(out [B,T,H,dv], hT [B,H,dk,dv] float32)``.  ``hT`` may be
    ``h0`` to update the state in place.
    """
    if stream is None and out is None and hT is None:
        r = (_fast or _open_fast()).decay_fwd(q, k, v, decay, h0, lengths, scale)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, H, dk, dv, pq, pk, pv, pd, strides = _decay_begin(q, k, v, decay, 4, "delta_decay_fwd")
    B, T = q.shape[:2]
    ph = _optional(h0, "h0", (B, H, dk, dv), torch.float32, dev)
    pl = _optional(lengths, "lengths", (B,), torch.int32, dev)
    out = _output(out, "out", (B, T, H, dv), q.dtype, dev, stream)
    hT = _output(hT, "hT", (B, H, dk, dv), torch.float32, dev, stream)
    st = _on(dev, _lib().delta_decay_fwd)(pq, pk, pv, pd, ph, pl, out.data_ptr(), hT.data_ptr(), B, T, H,
        dk, dv, strides, scale, code, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return out, hT


def delta_decay_step(q, k, v, decay, state, *, scale=1.0, out=None, stream=None):
    """One token of the same: q, k [B,H,dk], v [B,H,dv] (strides above the last axis as
    they are), state [B,H,dk,dv] float32 updated in place.  Returns out [B,H,dv]."""
    if stream is None and out is None:
        r = (_fast or _open_fast()).decay_step(q, k, v, decay, state, scale)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, H, dk, dv, pq, pk, pv, pd, strides = _decay_begin(q, k, v, decay, 3, "delta_decay_step")
    B = q.shape[0]
    ps = _tensor(state, "state", (B, H, dk, dv), torch.float32, dev)
    out = _output(out, "out", (B, H, dv), q.dtype, dev, stream)
    st = _on(dev, _lib().delta_decay_step)(pq, pk, pv, pd, ps, out.data_ptr(), B, H, dk, dv, strides, scale,
        code, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return out


def delta_decay_bwd(q, k, v, decay, dout, h0=None, dhT=None, *, scale=1.0, lengths=None, stream=None):
    """Gradients of ``delta_decay_fwd``: its arguments, dout [B,T,H,dv] contiguous and
    dhT [B,H,dk,dv] float32 or None.  Returns ``(dq, dk, dv, dh0)``, the first three in
    q's type and contiguous, dh0 float32.  The decays are constants and have none."""
    if stream is None:
        r = (_fast or _open_fast()).decay_bwd(q, k, v, decay, dout, h0, dhT, lengths, scale)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, H, dk, dv, pq, pk, pv, pd, strides = _decay_begin(q, k, v, decay, 4, "delta_decay_bwd")
    B, T = q.shape[:2]
    po = _tensor(dout, "dout", (B, T, H, dv), q.dtype, dev)
    ph = _optional(h0, "h0", (B, H, dk, dv), torch.float32, dev)
    pt = _optional(dhT, "dhT", (B, H, dk, dv), torch.float32, dev)
    pl = _optional(lengths, "lengths", (B,), torch.int32, dev)
    gq, gk = (_empty((B, T, H, dk), q.dtype, dev, stream) for _ in range(2))
    gv = _empty((B, T, H, dv), q.dtype, dev, stream)
    dh0 = _empty((B, H, dk, dv), torch.float32, dev, stream)
    st = _on(dev, _lib().delta_decay_bwd)(pq, pk, pv, pd, ph, pl, po, pt, gq.data_ptr(), gk.data_ptr(),
        gv.data_ptr(), dh0.data_ptr(), B, T, H, dk, dv, strides, scale, code, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return gq, gk, gv, dh0


def _rows(t, name, shape, dtype, dev):
    """A tensor [..., D] as rows: pointer and row stride.  Leading axes must
    fold into one."""
    p = _tensor(t, name, shape, dtype, dev, True)
    if t.dim() <= 2:
        return p, t.stride(0) if t.dim() == 2 else t.shape[-1]
    if not t.is_contiguous():
        t = t.flatten(0, -2) if _folds(t) else None
        if t is None:
            raise ValueError(f"the leading axes of {name} must fold into one row axis")
        return p, t.stride(0)
    return p, t.shape[-1]


def _folds(t):
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    return all(s == n2 * s2 for (_, s), (n2, s2) in zip(axes, axes[1:]))


def _weight(weight, D, dt, dev, name="weight"):
    wdt = weight.dtype if isinstance(weight, torch.Tensor) else None
    if wdt not in _CODES:
        raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
    return _tensor(weight, name, (D,), wdt, dev), _CODES[wdt]


def _per_row(shape, empty_value, D, dev, stream):
    """A float32 a row; rows without elements are never reached by the kernels."""
    t = _empty(shape, torch.float32, dev, stream)
    if D == 0:
        with torch.cuda.stream(stream):  # (None: the current one)
            t.fill_(empty_value)
    return t


def _norm_begin(x, weight, residual, name):
    code, dev = _begin(x, name, 0)
    if x.dim() < 1:
        raise ValueError("x must have at least one axis")
    D = x.shape[-1]
    px, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    pr, ldr = (None, D) if residual is None else _rows(residual, "residual", x.shape, x.dtype, dev)
    pw, wcode = _weight(weight, D, x.dtype, dev)
    rows = x.numel() // D if D else 0
    return code, dev, D, rows, px, ldx, pr, ldr, pw, wcode


def delta_add_rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, sum_out=None, stream=None):
    """``t = x + residual``, ``y = t * rsqrt(mean t^2 + eps) * weight`` over the
    last axis (at most 8192 wide).

    x, residual [..., D] bfloat16 or float32 (rows may be strided), weight [D]
    float32 or bfloat16.  Returns ``(y, sum, rstd)``: y in x's type, sum = t
    rounded to it (x itself without a residual), rstd [...] float32.
    ``sum_out`` may be ``x`` or ``residual`` to update the stream in place.
    """
    if stream is None and sum_out is None:
        r = (_fast or _open_fast()).norm_fwd(x, weight, residual, eps, False)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, D, rows, px, ldx, pr, ldr, pw, wcode = _norm_begin(x, weight, residual,
                                                                 "delta_add_rmsnorm_fwd")
    y = _empty(x.shape, x.dtype, dev, stream)
    rstd = _per_row(x.shape[:-1], eps ** -0.5 if eps > 0 else 0.0, D, dev, stream)
    if residual is not None:
        sum_out = _output(sum_out, "sum_out", x.shape, x.dtype, dev, stream)
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual: without one the sum is x")
    st = _on(dev, _lib().delta_add_rmsnorm_fwd)(px, pr, pw, y.data_ptr(),
        None if sum_out is None else sum_out.data_ptr(), rstd.data_ptr(), rows, D, ldx, ldr, eps,
        code, wcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return y, (x if sum_out is None else sum_out), rstd


def delta_add_rmsnorm_quant(x, weight, residual=None, *, eps=1e-6, sum_out=None, stream=None):
    """The same with y in e4m3 and one float32 scale a row (max |y| / 448; 1
    for a row of zeros).  Returns ``(y float8_e4m3fn, scale [...], sum)``."""
    if stream is None and sum_out is None:
        r = (_fast or _open_fast()).norm_fwd(x, weight, residual, eps, True)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, D, rows, px, ldx, pr, ldr, pw, wcode = _norm_begin(x, weight, residual,
                                                                 "delta_add_rmsnorm_quant")
    y = _empty(x.shape, E4M3, dev, stream)
    scale = _per_row(x.shape[:-1], 1.0, D, dev, stream)
    if residual is not None:
        sum_out = _output(sum_out, "sum_out", x.shape, x.dtype, dev, stream)
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual: without one the sum is x")
    st = _on(dev, _lib().delta_add_rmsnorm_quant)(px, pr, pw, y.data_ptr(), scale.data_ptr(),
        None if sum_out is None else sum_out.data_ptr(), rows, D, ldx, ldr, eps, code, wcode,
        _raw_stream(dev, stream))
    if st:
        _raise(st)
    return y, scale, (x if sum_out is None else sum_out)


def delta_add_rmsnorm_bwd(dy, sum, weight, rstd, dsum=None, *, dx=None, stream=None):
    """Gradients of ``delta_add_rmsnorm_fwd``: dy and the forward's sum [..., D]
    (contiguous, one type), rstd, and dsum, the gradient that arrives at sum,
    or None.  Returns ``(dx, dweight)``: dx (of x and of residual alike) in
    dy's type, dweight [D] float32.  ``dx`` may be ``dy`` or ``dsum``."""
    if stream is None and dx is None:
        r = (_fast or _open_fast()).norm_bwd(dy, sum, weight, rstd, dsum)
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(dy, "delta_add_rmsnorm_bwd", 0, "dy")
    if dy.dim() < 1:
        raise ValueError("dy must have at least one axis")
    D = dy.shape[-1]
    py = _tensor(dy, "dy", dy.shape, dy.dtype, dev)
    ps = _tensor(sum, "sum", dy.shape, dy.dtype, dev)
    pd = _optional(dsum, "dsum", dy.shape, dy.dtype, dev)
    pr = _tensor(rstd, "rstd", dy.shape[:-1], torch.float32, dev)
    pw, wcode = _weight(weight, D, dy.dtype, dev)
    dx = _output(dx, "dx", dy.shape, dy.dtype, dev, stream)
    dweight = _empty((D,), torch.float32, dev, stream)
    st = _on(dev, _lib().delta_add_rmsnorm_bwd)(py, ps, pw, pr, pd, dx.data_ptr(),
        dweight.data_ptr(), dy.numel() // D if D else 0, D, code, wcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return dx, dweight


def delta_add_layernorm_fwd(x, weight, bias=None, residual=None, *, eps=1e-5, sum_out=None, stream=None):
    """``t = x + residual``, ``y = (t - mean) * rsqrt(var + eps) * weight + bias`` over the
    last axis (at most 8192 wide), mean and var those of the row.

    x, residual [..., D] bfloat16 or float32 (rows may be strided), weight and bias
    [D] float32 or bfloat16.  Returns ``(y, sum, mean, rstd)``: y in x's type, sum = t
    rounded to it (x itself without a residual), mean and rstd [...] float32.
    ``sum_out`` may be ``x`` or ``residual`` to update the stream in place.
    """
    if stream is None and sum_out is None:
        r = (_fast or _open_fast()).layernorm_fwd(x, weight, bias, residual, eps)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, D, rows, px, ldx, pr, ldr, pw, wcode = _norm_begin(x, weight, residual,
                                                                 "delta_add_layernorm_fwd")
    pb, bcode = (None, 0) if bias is None else _weight(bias, D, x.dtype, dev, "bias")
    y = _empty(x.shape, x.dtype, dev, stream)
    mean = _per_row(x.shape[:-1], 0.0, D, dev, stream)
    rstd = _per_row(x.shape[:-1], eps ** -0.5 if eps > 0 else 0.0, D, dev, stream)
    if residual is not None:
        sum_out = _output(sum_out, "sum_out", x.shape, x.dtype, dev, stream)
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual: without one the sum is x")
    st = _on(dev, _lib().delta_add_layernorm_fwd)(px, pr, pw, pb, y.data_ptr(),
        None if sum_out is None else sum_out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, D, ldx,
        ldr, eps, code, wcode, bcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return y, (x if sum_out is None else sum_out), mean, rstd


def delta_add_layernorm_bwd(dy, sum, weight, mean, rstd, dsum=None, *, dx=None, stream=None):
    """Gradients of ``delta_add_layernorm_fwd``: dy and the forward's sum [..., D]
    (contiguous, one type), mean and rstd, and dsum, the gradient that arrives at sum,
    or None.  Returns ``(dx, dweight, dbias)``: dx (of x and of residual alike) in
    dy's type, dweight and dbias [D] float32.  ``dx`` may be ``dy`` or ``dsum``."""
    if stream is None and dx is None:
        r = (_fast or _open_fast()).layernorm_bwd(dy, sum, weight, mean, rstd, dsum)
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(dy, "delta_add_layernorm_bwd", 0, "dy")
    if dy.dim() < 1:
        raise ValueError("dy must have at least one axis")
    D = dy.shape[-1]
    py = _tensor(dy, "dy", dy.shape, dy.dtype, dev)
    ps = _tensor(sum, "sum", dy.shape, dy.dtype, dev)
    pd = _optional(dsum, "dsum", dy.shape, dy.dtype, dev)
    pm = _tensor(mean, "mean", dy.shape[:-1], torch.float32, dev)
    pr = _tensor(rstd, "rstd", dy.shape[:-1], torch.float32, dev)
    pw, wcode = _weight(weight, D, dy.dtype, dev)
    dx = _output(dx, "dx", dy.shape, dy.dtype, dev, stream)
    dweight, dbias = (_empty((D,), torch.float32, dev, stream) for _ in range(2))
    st = _on(dev, _lib().delta_add_layernorm_bwd)(py, ps, pw, pm, pr, pd, dx.data_ptr(), dweight.data_ptr(),
        dbias.data_ptr(), dy.numel() // D if D else 0, D, code, wcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return dx, dweight, dbias


def _linear_begin(x, w, bias, residual, act, dtype, odt, dev):
    """shared checks: sizes, pointers and row strides of a linear layer"""
    acode = _ACTS.get(act)
    if acode is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or x.dim() < 1:
        raise ValueError("x must be [..., K] and w [N, K]")
    N, K = w.shape
    px, ldx = _rows(x, "x", x.shape[:-1] + (K,), dtype, dev)
    pw = _tensor(w, "w", w.shape, dtype, dev, True)
    pb, bcode = (None, 0) if bias is None else _weight(bias, N, odt, dev, "bias")
    shape = x.shape[:-1] + (N,)
    pr, ldr = (None, N) if residual is None else _rows(residual, "residual", shape, odt, dev)
    M = 1
    for n in x.shape[:-1]:
        M *= n
    _within_int("the layer", (M, N, K))
    return acode, M, N, K, px, ldx, pw, w.stride(0), pb, bcode, pr, ldr, shape


def delta_linear_fwd(x, w, bias=None, residual=None, *, act="none", save_pre=False, out=None,
                     stream=None):
    """``out = act(x w^T + bias) + residual``, finished in float32.

    x [..., K] and w [N, K] bfloat16 or float32 (rows may be strided), bias [N]
    float32 or bfloat16, residual [..., N] in x's type; ``act`` is "none",
    "silu" or "gelu" (tanh form).  Returns out [..., N], with ``save_pre``
    ``(out, pre)`` for ``delta_linear_bwd``.  ``out`` may be ``residual``.
    """
    if stream is None and out is None:
        r = (_fast or _open_fast()).linear_fwd(x, w, bias, residual, _ACTS.get(act, -1), save_pre)
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(x, "delta_linear_fwd", 0)
    dt = x.dtype
    acode, M, N, K, px, ldx, pw, ldw, pb, bcode, pr, ldr, shape = _linear_begin(
        x, w, bias, residual, act, dt, dt, dev)
    out = _output(out, "out", shape, dt, dev, stream)
    pre = _empty(shape, dt, dev, stream) if save_pre else None
    st = _on(dev, _lib().delta_linear_fwd)(px, pw, pb, pr, out.data_ptr(),
        None if pre is None else pre.data_ptr(), M, N, K, ldx, ldw, ldr, acode, code, bcode,
        _raw_stream(dev, stream))
    if st:
        _raise(st)
    return (out, pre) if save_pre else out


def delta_linear_quant(x, x_scale, w, w_scale, bias=None, residual=None, *, act="none", out=None,
                       stream=None):
    """The same with x [..., K] and w [N, K] in float8_e4m3fn and a float32 scale
    for each of their rows, x_scale [...] and w_scale [N]; residual and out are
    bfloat16."""
    if stream is None and out is None:
        r = (_fast or _open_fast()).linear_quant(x, x_scale, w, w_scale, bias, residual,
                                                 _ACTS.get(act, -1))
        if r is not NotImplemented:
            return _checked(r)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("delta_linear_quant needs CUDA tensors")
    acode, M, N, K, px, ldx, pw, ldw, pb, bcode, pr, ldr, shape = _linear_begin(
        x, w, bias, residual, act, E4M3, torch.bfloat16, dev)
    psx = _tensor(x_scale, "x_scale", x.shape[:-1], torch.float32, dev)
    psw = _tensor(w_scale, "w_scale", (N,), torch.float32, dev)
    out = _output(out, "out", shape, torch.bfloat16, dev, stream)
    st = _on(dev, _lib().delta_linear_quant)(px, psx, pw, psw, pb, pr, out.data_ptr(), M, N, K, ldx,
        ldw, ldr, acode, bcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return out


def delta_linear_bwd(x, w, dout, pre=None, *, act="none", want=(True, True, True), stream=None):
    """Gradients of ``delta_linear_fwd``: x and w as there, dout and pre [..., N]
    contiguous (pre only with an activation).  Returns ``(dx, dw, dbias)``, dx
    and dw in x's type, dbias float32; those not wanted are None."""
    if stream is None:
        r = (_fast or _open_fast()).linear_bwd(x, w, dout, pre, _ACTS.get(act, -1), *want)
        if r is not NotImplemented:
            return _checked(r)
    code, dev = _begin(x, "delta_linear_bwd", 0)
    dt = x.dtype
    acode, M, N, K, px, ldx, pw, ldw, _, _, _, _, shape = _linear_begin(
        x, w, None, None, act, dt, dt, dev)
    po = _tensor(dout, "dout", shape, dt, dev)
    pp = _tensor(pre, "pre", shape, dt, dev) if acode or pre is not None else None
    dx = _empty(x.shape, dt, dev, stream) if want[0] else None
    dw = _empty((N, K), dt, dev, stream) if want[1] else None
    db = _empty((N,), torch.float32, dev, stream) if want[2] else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = _on(dev, _lib().delta_linear_bwd)(px, pw, po, pp, ptr(dx), ptr(dw), ptr(db), M, N, K, ldx,
        ldw, acode, code, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return dx, dw, db


def _glu_begin(x, w, act, name):
    """shared checks: sizes, pointers and row strides of a gated layer"""
    code, dev = _begin(x, name, 0)
    if isinstance(w, torch.Tensor) and w.dim() == 2 and w.shape[0] % 2:
        raise ValueError(f"w must have two halves of rows, got {w.shape[0]}")
    acode, M, N, K, px, ldx, pw, ldw, _, _, _, _, shape = _linear_begin(x, w, None, None, act, x.dtype, x.dtype, dev)
    return code, dev, acode, M, N // 2, K, px, ldx, pw, ldw, shape


def delta_glu_fwd(x, w, bias=None, *, act="silu", save_pre=False, out=None, stream=None):
    """The first half of a gated feed-forward layer: ``out = act(g) * u`` with
    ``(g, u) = x w^T + bias``, finished in float32.

    x [..., K] and w [2 N, K] bfloat16 or float32 (rows may be strided): N rows for the
    gate, then N for the other projection; bias [2 N] float32 or bfloat16; ``act`` as in
    ``delta_linear_fwd``.  Returns out [..., N], with ``save_pre`` ``(out, pre [..., 2 N])``
    for ``delta_glu_bwd``.
    """
    if stream is None and out is None:
        r = (_fast or _open_fast()).glu_fwd(x, w, bias, _ACTS.get(act, -1), save_pre)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, acode, M, N, K, px, ldx, pw, ldw, shape = _glu_begin(x, w, act, "delta_glu_fwd")
    pb, bcode = (None, 0) if bias is None else _weight(bias, 2 * N, x.dtype, dev, "bias")
    out = _output(out, "out", shape[:-1] + (N,), x.dtype, dev, stream)
    pre = _empty(shape, x.dtype, dev, stream) if save_pre else None
    st = _on(dev, _lib().delta_glu_fwd)(px, pw, pb, out.data_ptr(), None if pre is None else pre.data_ptr(),
        M, N, K, ldx, ldw, acode, code, bcode, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return (out, pre) if save_pre else out


def delta_glu_bwd(x, w, dout, pre, *, act="silu", want=(True, True, True), stream=None):
    """Gradients of ``delta_glu_fwd``: x and w as there, dout [..., N] and pre [..., 2 N]
    contiguous.  Returns ``(dx, dw, dbias)``, dx and dw in x's type, dbias float32; those
    not wanted are None."""
    if stream is None:
        r = (_fast or _open_fast()).glu_bwd(x, w, dout, pre, _ACTS.get(act, -1), *want)
        if r is not NotImplemented:
            return _checked(r)
    code, dev, acode, M, N, K, px, ldx, pw, ldw, shape = _glu_begin(x, w, act, "delta_glu_bwd")
    dt = x.dtype
    po = _tensor(dout, "dout", shape[:-1] + (N,), dt, dev)
    pp = _tensor(pre, "pre", shape, dt, dev)
    dx = _empty(x.shape, dt, dev, stream) if want[0] else None
    dw = _empty((2 * N, K), dt, dev, stream) if want[1] else None
    db = _empty((2 * N,), torch.float32, dev, stream) if want[2] else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = _on(dev, _lib().delta_glu_bwd)(px, pw, po, pp, ptr(dx), ptr(dw), ptr(db), M, N, K, ldx, ldw, acode,
        code, _raw_stream(dev, stream))
    if st:
        _raise(st)
    return dx, dw, db
