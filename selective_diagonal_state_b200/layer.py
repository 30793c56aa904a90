"""The operators around the mixer, on torch CUDA tensors: RMS norm with the residual's
addition and 8-bit output, rotary positions, and linear attention with a decay a head.

As in ``scan.py``, torch serves for device memory and streams only: the helpers check the
tensors, allocate outputs (``out`` / the named buffers take the caller's), build the
descriptor from sizes and strides and make one call of the C ABI (``include/ssm_scan.h``
says what each computes).  Tensors may have any strides with a dense last dimension.  Calls
go to ``stream`` (default: the current stream of the tensors' device, made current for the
call where it is not).  Workspaces come from torch's allocator on that stream unless
given; calls that overlap on the GPU, captured graphs among them, must not share one.
"""
from __future__ import annotations

import dataclasses

import torch

from . import abi

_DTYPES = {torch.bfloat16: abi.DTYPE_BF16, torch.float32: abi.DTYPE_F32}
_QUANT = {None: abi.QUANT_NONE, "row": abi.QUANT_ROW, "block": abi.QUANT_BLOCK}
_LAYOUT = {"half": abi.ROPE_HALF, "pairs": abi.ROPE_PAIRS}
_SCALING = {"plain": abi.ROPE_PLAIN, "linear": abi.ROPE_LINEAR, "ntk": abi.ROPE_NTK,
            "bands": abi.ROPE_BANDS}
QUANT_BLOCK_COLUMNS = 128


class _Call:
    """The device and stream of a call: ``tensors`` all live on ``first``'s device, which is
    current inside, as is ``stream`` where one is given (torch's allocations inside are its)."""

    def __init__(self, stream, first, *tensors):
        if not first.is_cuda:
            raise ValueError("every tensor must live on a CUDA device (no CPU path)")
        dev = first.get_device()
        for t in tensors:
            if t is not None and (not t.is_cuda or t.get_device() != dev):
                raise ValueError("the tensors of a call must share one CUDA device")
        self.guards = []
        if torch.cuda.current_device() != dev:
            self.guards.append(torch.cuda.device(dev))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=dev)
            if stream.device_index != dev:
                raise ValueError("the stream belongs to another device than the tensors")
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _want(t, name, shape, dtype, dense=False):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has type {t.dtype}, expected {dtype}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not dense and t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be dense")


def _io(t, name):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} has type {t.dtype}; bfloat16 and float32 are supported")
    return _DTYPES[t.dtype]


def _workspace(nbytes, given, device):
    if given is not None:
        return given, given.numel() * given.element_size()
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


# ---- RMS norm --------------------------------------------------------------------------

@dataclasses.dataclass
class Normed:
    """``r`` the residual stream (``x`` itself without a residual), ``y`` the norm in the I/O
    type, ``y8`` its e4m3 codes with fp32 ``scales`` ([..., 1] or [..., dim / 128]), ``rstd``
    what the backward reads; None what was not asked for."""

    r: object
    y: object = None
    y8: object = None
    scales: object = None
    rstd: object = None


def _rows(t, name, dim):
    """Row stride of [..., dim] seen as evenly spaced rows."""
    step = n = None
    for size, stride in zip(t.shape[-2::-1], t.stride()[-2::-1]):
        if size == 1:
            continue
        if step is None:
            step, n = stride, size
        elif stride == n * step:
            n *= size
        else:
            raise ValueError(f"the rows of {name} must be evenly spaced")
    return dim if step is None else step


def _norm_desc(like, dim, eps, quant, **strides):
    d = abi.RmsnormDesc()
    d.rows, d.dim = like.numel() // dim if dim else 0, dim
    d.eps, d.dtype_io, d.quant = eps, _io(like, "x"), quant
    for k, t in strides.items():
        setattr(d, "stride_" + k, dim if t is None else _rows(t, k, dim))
    return d


def rmsnorm(x, weight=None, residual=None, eps=1e-5, quant=None, want_y=None, want_rstd=False,
            r=None, stream=None) -> Normed:
    """RMS norm of ``x`` (+ ``residual``) over its last dimension; the rows of every tensor,
    whatever their leading dimensions, are evenly spaced.

    ``quant``: None, "row" or "block" (128 columns) for e4m3 codes with scales; ``want_y``: also
    the unquantised norm (default: only without ``quant``); ``want_rstd`` for a later
    :func:`rmsnorm_backward`; ``r``: where the sum goes (may be ``x`` or ``residual``)."""
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'row' or 'block', not {quant!r}")
    dim, dt, shape = x.shape[-1], x.dtype, x.shape
    _want(x, "x", shape, dt)
    if weight is not None:
        _want(weight, "weight", (dim,), torch.float32, True)
    if residual is not None:
        _want(residual, "residual", shape, dt)
    if r is not None:
        _want(r, "r", shape, dt)
    want_y = quant is None if want_y is None else want_y
    if quant is None and not want_y:
        raise ValueError("without quant the norm itself is the output: want_y cannot be False")
    with _Call(stream, x, weight, residual, r) as st:
        if r is None and residual is not None:
            r = torch.empty(shape, dtype=dt, device=x.device)
        out = Normed(r=x if r is None else r)
        if want_y:
            out.y = torch.empty(shape, dtype=dt, device=x.device)
        if quant is not None:
            out.y8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
            blocks = dim // QUANT_BLOCK_COLUMNS if quant == "block" else 1
            out.scales = torch.empty(*shape[:-1], blocks, dtype=torch.float32, device=x.device)
        if want_rstd:
            out.rstd = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        d = _norm_desc(x, dim, eps, _QUANT[quant], x=x, residual=residual, r=r, y=out.y, y8=out.y8)
        abi.ssm_rmsnorm_fwd(d, x, residual, weight, r, out.y, out.y8, out.scales, out.rstd, st)
    return out


def rmsnorm_backward(dy, r, weight, rstd, dr=None, dx=None, want_dweight=None, workspace=None,
                     stream=None):
    """(dx, dweight) for ``dy``, the gradient of the norm, and ``dr``, that of the residual
    stream behind it; ``r`` and ``rstd`` as :func:`rmsnorm` returned them.  dx is the gradient
    of ``x`` and of ``residual``; dweight (fp32) is None without a weight."""
    dim, dt, shape = r.shape[-1], r.dtype, r.shape
    _want(r, "r", shape, dt)
    _want(dy, "dy", shape, dt)
    _want(rstd, "rstd", shape[:-1], torch.float32, True)
    if weight is not None:
        _want(weight, "weight", (dim,), torch.float32, True)
    if dr is not None:
        _want(dr, "dr", shape, dt)
    if dx is not None:
        _want(dx, "dx", shape, dt)
    want_dweight = weight is not None if want_dweight is None else want_dweight
    with _Call(stream, r, dy, weight, rstd, dr, dx, workspace) as st:
        if dx is None:
            dx = torch.empty(shape, dtype=dt, device=r.device)
        dw = torch.empty(dim, dtype=torch.float32, device=r.device) if want_dweight else None
        d = _norm_desc(r, dim, 0.0, abi.QUANT_NONE, dy=dy, r=r, dr=dr, dx=dx)
        ws, n = None, 0
        if want_dweight:
            ws, n = _workspace(abi.ssm_rmsnorm_workspace_size(d), workspace, r.device)
        abi.ssm_rmsnorm_bwd(d, dy, r, weight, rstd, dr, dx, dw, ws, n, st)
    return dx, dw


# ---- rotary positions ------------------------------------------------------------------

def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, low_turns=1.0,
                     high_turns=4.0, original_context=0.0, device="cuda"):
    """fp64 [rot_dim / 2] frequencies (radians a position) on ``device``.

    ``scaling``: "plain"; "linear" (positions interpolated by ``factor``); "ntk" (a larger
    base); "bands" (pairs that turn often within ``original_context`` positions are kept,
    those that turn seldom interpolated, a linear blend between)."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {sorted(_SCALING)}, not {scaling!r}")
    f = abi.ssm_rope_frequencies(rot_dim, base, _SCALING[scaling], factor, low_turns, high_turns,
                                 original_context)
    return torch.tensor(f, dtype=torch.float64, device=device)


def _rope(call, q, k, freq, positions, layout, magnitude, q_out, k_out, stream):
    if layout not in _LAYOUT:
        raise ValueError(f"layout must be 'half' or 'pairs', not {layout!r}")
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k are both None")
    if first.dim() != 4:
        raise ValueError(f"q and k are [batch, seqlen, heads, headdim], not {tuple(first.shape)}")
    b, L, _, dim = first.shape
    d = abi.RopeDesc()
    d.batch, d.seqlen, d.headdim, d.rot_dim = b, L, dim, 2 * freq.numel()
    d.magnitude, d.layout, d.dtype_io = magnitude, _LAYOUT[layout], _io(first, "q")
    _want(freq, "freq", (freq.numel(),), torch.float64, True)
    if positions is not None:
        if positions.dtype != torch.int64 or tuple(positions.shape) not in ((b, L), (L,)):
            raise ValueError("positions must be int64 [batch, seqlen] or [seqlen]")
        if positions.dim() == 1:
            d.stride_pos[:] = 0, positions.stride(0)
        else:
            d.stride_pos[:] = positions.stride()
    outs = []
    with _Call(stream, first, q, k, freq, positions, q_out, k_out) as st:
        for name, x, y in (("q", q, q_out), ("k", k, k_out)):
            if x is None:
                if y is not None:
                    raise ValueError(f"an output without its input: {name}")
                outs.append(None)
                continue
            _want(x, name, (b, L, x.shape[2] if x.dim() == 4 else -1, dim), first.dtype)
            if y is None:
                y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            _want(y, name + "_out", x.shape, x.dtype)
            setattr(d, "nheads_" + name, x.shape[2])
            getattr(d, "stride_" + name)[:] = x.stride()[:3]
            getattr(d, f"stride_{name}_out")[:] = y.stride()[:3]
            outs.append(y)
        call(d, q, k, freq, positions, outs[0], outs[1], st)
    return tuple(outs)


def rope(q, k, freq, positions=None, layout="half", magnitude=1.0, q_out=None, k_out=None,
         stream=None):
    """(q, k) with rotary positions on the first ``2 * len(freq)`` values of each head.

    q, k: [batch, seqlen, heads, headdim] (either may be None); ``freq`` from
    :func:`rope_frequencies`; ``positions``: int64 [batch, seqlen] or [seqlen] (default 0, 1, ...);
    ``layout``: "half" pairs value i with i + rot / 2, "pairs" neighbours; outputs may be the inputs."""
    return _rope(abi.ssm_rope_fwd, q, k, freq, positions, layout, magnitude, q_out, k_out, stream)


def rope_backward(dq, dk, freq, positions=None, layout="half", magnitude=1.0, dq_out=None,
                  dk_out=None, stream=None):
    """Gradients of :func:`rope`'s inputs for those of its outputs."""
    return _rope(abi.ssm_rope_bwd, dq, dk, freq, positions, layout, magnitude, dq_out, dk_out,
                 stream)


# ---- linear attention ------------------------------------------------------------------

def _la_desc(q, k, v, log_decay, lengths, scale, route, **more):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are [batch, seqlen, heads, headdim]")
    b, L, h, dk = q.shape
    g, dv = k.shape[2], v.shape[3]
    _want(q, "q", q.shape, q.dtype)
    _want(k, "k", (b, L, g, dk), q.dtype)
    _want(v, "v", (b, L, g, dv), q.dtype)
    _want(log_decay, "log_decay", (h,), torch.float32, True)
    if lengths is not None:
        _want(lengths, "lengths", (b,), torch.int32, True)
    d = abi.LinattnDesc()
    d.batch, d.seqlen, d.nheads, d.nheads_kv, d.dim_k, d.dim_v = b, L, h, g, dk, dv
    d.scale, d.dtype_io, d.route = dk ** -0.5 if scale is None else scale, _io(q, "q"), route
    d.stride_q[:], d.stride_k[:], d.stride_v[:] = q.stride()[:3], k.stride()[:3], v.stride()[:3]
    for name, (t, shape) in more.items():
        _want(t, name, shape, q.dtype)
        getattr(d, "stride_" + name)[:] = t.stride()[:3]
    return d


def linattn(q, k, v, log_decay, scale=None, state=None, lengths=None, out=None, want_state=True,
            state_out=None, route=abi.LINATTN_AUTO, workspace=None, stream=None):
    """(o, state): linear attention with the decay e^log_decay[h] a head, over whole sequences.

    q [B, L, H, dim_k], k [B, L, G, dim_k], v [B, L, G, dim_v] with H a multiple of G;
    ``scale`` defaults to dim_k ** -0.5; ``state`` fp32 [B, H, dim_k, dim_v] enters (default
    zero); ``lengths`` int32 [B]: rows behind them are neither read nor written (``out``
    keeps them).  ``state_out`` takes the final state (may be ``state``)."""
    b, L, h = q.shape[:3]
    shape = (b, h, q.shape[3], v.shape[3])
    for name, s in (("state", state), ("state_out", state_out)):
        if s is not None:
            _want(s, name, shape, torch.float32, True)
    with _Call(stream, q, k, v, log_decay, state, lengths, out, state_out, workspace) as st:
        if out is None:
            out = torch.empty(b, L, h, v.shape[3], dtype=q.dtype, device=q.device)
        if state_out is None and want_state:
            state_out = torch.empty(shape, dtype=torch.float32, device=q.device)
        d = _la_desc(q, k, v, log_decay, lengths, scale, route, o=(out, (b, L, h, v.shape[3])))
        ws, n = _workspace(abi.ssm_linattn_workspace_size(d, abi.PASS_FWD), workspace, q.device)
        abi.ssm_linattn_fwd(d, q, k, v, log_decay, state, lengths, out, state_out, ws, n, st)
    return out, state_out


def linattn_backward(q, k, v, log_decay, do, scale=None, state=None, dstate=None, lengths=None,
                     out=None, route=abi.LINATTN_AUTO, workspace=None, stream=None):
    """(dq, dk, dv, dstate): gradients of :func:`linattn` for ``do`` and ``dstate``, that of the
    final state (default zero); the returned dstate is that of the entering ``state``.
    ``out``: buffers (dq, dk, dv), whose rows behind ``lengths`` stay as they are."""
    b, L, h = q.shape[:3]
    shape = (b, h, q.shape[3], v.shape[3])
    for name, s in (("state", state), ("dstate", dstate)):
        if s is not None:
            _want(s, name, shape, torch.float32, True)
    dq, dk, dv = out if out is not None else (None, None, None)
    with _Call(stream, q, k, v, log_decay, do, state, dstate, lengths, dq, dk, dv, workspace) as st:
        dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) if y is None else y
                      for x, y in ((q, dq), (k, dk), (v, dv)))
        din = torch.empty(shape, dtype=torch.float32, device=q.device)
        d = _la_desc(q, k, v, log_decay, lengths, scale, route, o=(do, (b, L, h, v.shape[3])),
                     dq=(dq, q.shape), dk=(dk, k.shape), dv=(dv, v.shape))
        ws, n = _workspace(abi.ssm_linattn_workspace_size(d, abi.PASS_BWD), workspace, q.device)
        abi.ssm_linattn_bwd(d, q, k, v, log_decay, state, lengths, do, dstate, dq, dk, dv, din, ws,
                            n, st)
    return dq, dk, dv, din


def linattn_step(q, k, v, log_decay, state, scale=None, out=None, stream=None):
    """o [B, 1, H, dim_v] of one token (seqlen 1); ``state`` is updated in place."""
    b, L, h = q.shape[:3]
    _want(state, "state", (b, h, q.shape[3], v.shape[3]), torch.float32, True)
    with _Call(stream, q, k, v, log_decay, state, out) as st:
        if out is None:
            out = torch.empty(b, L, h, v.shape[3], dtype=q.dtype, device=q.device)
        d = _la_desc(q, k, v, log_decay, None, scale, abi.LINATTN_AUTO,
                     o=(out, (b, L, h, v.shape[3])))
        abi.ssm_linattn_step(d, q, k, v, log_decay, state, out, st)
    return out
