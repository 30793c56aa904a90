"""The operators around the mixer, on torch CUDA tensors: RMS norm with the residual's
addition and 8-bit output, rotary positions, and linear attention with a decay a head.

As in ``scan.py``, torch serves for device memory and streams only: the helpers check the
tensors, allocate outputs (``out`` / the named buffers take the caller's) and make one call
of the C ABI (``include/ssm_scan.h`` says what each computes).  Tensors may have any strides
with a dense last dimension.  Calls go to ``stream`` (default: the current stream of the
tensors' device, made current for the call where it is not).  Workspaces come from torch's
allocator on that stream unless given; calls that overlap on the GPU, captured graphs among
them, must not share one.

What a call checks and derives from its tensors' shapes, strides and types (never from their
contents or addresses) is kept for the next call with the same ones, once a call has gone
through: the checks alone would take longer than the smallest kernels.
"""
from __future__ import annotations

import contextlib
import dataclasses

import torch

from . import abi

_DTYPES = {torch.bfloat16: abi.DTYPE_BF16, torch.float32: abi.DTYPE_F32}
_QUANT = {None: abi.QUANT_NONE, "row": abi.QUANT_ROW, "block": abi.QUANT_BLOCK}
_LAYOUT = {"half": abi.ROPE_HALF, "pairs": abi.ROPE_PAIRS}
_SCALING = {"plain": abi.ROPE_PLAIN, "linear": abi.ROPE_LINEAR, "ntk": abi.ROPE_NTK,
            "bands": abi.ROPE_BANDS}
QUANT_BLOCK_COLUMNS = 128

_PLANS = {}
_MOST_PLANS = 1024
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Plan:
    """Descriptor, device and sizes of a call, from its tensors' layouts."""

    __slots__ = ("dev", "desc", "lib", "ws", "likes", "key")   # key: None once the plan is kept


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _like(shape, dtype, dev):
    """What ``torch.empty_like`` takes for a dense tensor of this shape (one value, expanded:
    a third of the time of ``torch.empty`` with its arguments)."""
    t = torch.empty((0,) if 0 in shape else (), dtype=dtype, device=dev)
    if type(t) is not torch.Tensor:     # a mode that makes tensors without memory is on
        raise ValueError("the tensors of a call must have memory on their device (no fake tensors)")
    return t.view(shape) if 0 in shape else t.expand(shape)    # (of nothing, the strides would stay 0)


_new = torch.empty_like


def _rows_of(like, lengths):
    """An output of which a call with ``lengths`` leaves rows unwritten: those are zeros."""
    return _new(like) if lengths is None else torch.zeros_like(like)


def _plan(key, make, *args):
    p = _PLANS.get(key)
    if p is None:
        p = make(*args)
        p.lib = abi.load_library()
        p.key = key
    return p


def _keep(p):
    if len(_PLANS) >= _MOST_PLANS:
        _PLANS.clear()
    key, p.key = p.key, None
    _PLANS[key] = p


def _device(first, *tensors):
    if not first.is_cuda:
        raise ValueError("every tensor must live on a CUDA device (no CPU path)")
    dev = first.get_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.get_device() != dev):
            raise ValueError("the tensors of a call must share one CUDA device")
    return dev


@contextlib.contextmanager
def _elsewhere(dev, stream):
    """Makes ``dev`` and ``stream`` current (torch's allocations inside are the stream's)."""
    with torch.cuda.device(dev):
        if stream is None:
            yield _raw_stream(dev)
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        if stream.device_index != dev:
            raise ValueError("the stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _on_device(go, p, stream, *args):
    """go(plan, raw stream, ...) on the plan's device and the caller's stream."""
    if stream is None and _current_device() == p.dev:
        out = go(p, _raw_stream(p.dev), *args)
    else:
        with _elsewhere(p.dev, stream) as st:
            out = go(p, st, *args)
    if p.key is not None:
        _keep(p)
    return out


def _ptr(t):
    return None if t is None else t.data_ptr()


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


def _workspace(p, given):
    """(address, bytes, what keeps it alive)"""
    if given is not None:
        if given.get_device() != p.dev:
            raise ValueError("the workspace must live on the tensors' device")
        if not given.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if p.ws == 0:
        return None, 0, None
    w = torch.empty(p.ws, dtype=torch.uint8, device=p.dev)
    return w.data_ptr(), p.ws, w


def _dense_strides(shape):
    s, out = 1, []
    for n in reversed(shape):
        out.append(s)
        s *= max(n, 1)
    return tuple(reversed(out))


# ---- RMS norm --------------------------------------------------------------------------

@dataclasses.dataclass(slots=True)
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
    if t.numel() == 0:
        return dim
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


def _norm_plan(like, eps, quant, weight, dev, **tensors):
    """``like``: the tensor whose shape and type all others have; outputs not named are dense."""
    if like.dim() == 0:
        raise ValueError("the norm runs over a last dimension: x has none")
    dim = like.shape[-1]
    if weight is not None:
        _want(weight, "weight", (dim,), torch.float32, True)
    p = _Plan()
    p.dev, p.desc, p.ws = dev, abi.RmsnormDesc(), 0
    d = p.desc
    d.rows, d.dim = like.numel() // dim if dim else 0, dim
    d.eps, d.dtype_io, d.quant = eps, _io(like, "x"), quant
    for f, _ in abi.RmsnormDesc._fields_:
        if f.startswith("stride_"):
            t = tensors.get(f[7:])
            if t is not None:
                _want(t, f[7:], like.shape, like.dtype)
            setattr(d, f, dim if t is None else _rows(t, f[7:], dim))
    return p


def _norm_fwd_plan(x, weight, residual, r, eps, quant, want_y):
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'row' or 'block', not {quant!r}")
    if quant is None and want_y is False:
        raise ValueError("without quant the norm itself is the output: want_y cannot be False")
    dev = _device(x, weight, residual, r)
    p = _norm_plan(x, eps, _QUANT[quant], weight, dev, x=x, residual=residual, r=r)
    shape, io, y8, scales = x.shape, _like(x.shape, x.dtype, dev), None, None
    if quant is not None:
        y8 = _like(shape, torch.float8_e4m3fn, dev)
        scales = _like((*shape[:-1], shape[-1] // QUANT_BLOCK_COLUMNS if quant == "block" else 1), torch.float32, dev)
    want_y = quant is None if want_y is None else want_y
    p.likes = (io if residual is not None and r is None else None, io if want_y else None, y8, scales,
               _like(shape[:-1], torch.float32, dev))
    return p


def _norm_fwd(p, st, x, weight, residual, r, want_rstd):
    lr, ly, l8, ls, lrstd = p.likes
    if lr is not None:
        r = _new(lr)
    out = Normed(x if r is None else r, None if ly is None else _new(ly), None if l8 is None else _new(l8),
                 None if ls is None else _new(ls), _new(lrstd) if want_rstd else None)
    rc = p.lib.ssm_rmsnorm_fwd(p.desc, x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(r), _ptr(out.y),
                               _ptr(out.y8), _ptr(out.scales), _ptr(out.rstd), st)
    if rc:
        abi._check(rc, "ssm_rmsnorm_fwd")
    return out


def rmsnorm(x, weight=None, residual=None, eps=1e-5, quant=None, want_y=None, want_rstd=False,
            r=None, stream=None) -> Normed:
    """RMS norm of ``x`` (+ ``residual``) over its last dimension; the rows of every tensor,
    whatever their leading dimensions, are evenly spaced.

    ``quant``: None, "row" or "block" (128 columns) for e4m3 codes with scales; ``want_y``: also
    the unquantised norm (default: only without ``quant``); ``want_rstd`` for a later
    :func:`rmsnorm_backward`; ``r``: where the sum goes (may be ``x`` or ``residual`` itself)."""
    eps = float(eps)
    p = _plan(("norm", _sig(x), _sig(weight), _sig(residual), _sig(r), eps, quant, want_y),
              _norm_fwd_plan, x, weight, residual, r, eps, quant, want_y)
    return _on_device(_norm_fwd, p, stream, x, weight, residual, r, want_rstd)


def _norm_bwd_plan(dy, r, weight, rstd, dr, dx):
    dev = _device(r, dy, weight, rstd, dr, dx)
    _want(rstd, "rstd", r.shape[:-1], torch.float32, True)
    p = _norm_plan(r, 0.0, abi.QUANT_NONE, weight, dev, dy=dy, r=r, dr=dr, dx=dx)
    p.ws = abi.ssm_rmsnorm_workspace_size(p.desc)
    p.likes = _like(r.shape, r.dtype, dev), _like(r.shape[-1:], torch.float32, dev)
    return p


def _norm_bwd(p, st, dy, r, weight, rstd, dr, dx, want_dweight, workspace):
    if dx is None:
        dx = _new(p.likes[0])
    dw, ws, n, keep = None, None, 0, None
    if want_dweight:
        dw = _new(p.likes[1])
        ws, n, keep = _workspace(p, workspace)
    rc = p.lib.ssm_rmsnorm_bwd(p.desc, dy.data_ptr(), r.data_ptr(), _ptr(weight), rstd.data_ptr(),
                               _ptr(dr), dx.data_ptr(), _ptr(dw), ws, n, st)
    if rc:
        abi._check(rc, "ssm_rmsnorm_bwd")
    return dx, dw


def rmsnorm_backward(dy, r, weight, rstd, dr=None, dx=None, want_dweight=None, workspace=None,
                     stream=None):
    """(dx, dweight) for ``dy``, the gradient of the norm, and ``dr``, that of the residual
    stream behind it; ``r`` and ``rstd`` as :func:`rmsnorm` returned them; ``dx`` may be ``dy`` or ``dr``
    itself.  dx is the gradient
    of ``x`` and of ``residual``; dweight (fp32) is None without a weight."""
    p = _plan(("norm'", _sig(dy), _sig(r), _sig(weight), _sig(rstd), _sig(dr), _sig(dx)),
              _norm_bwd_plan, dy, r, weight, rstd, dr, dx)
    return _on_device(_norm_bwd, p, stream, dy, r, weight, rstd, dr, dx,
                      weight is not None if want_dweight is None else want_dweight, workspace)


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


def _rope_plan(q, k, freq, positions, layout, magnitude, q_out, k_out):
    if layout not in _LAYOUT:
        raise ValueError(f"layout must be 'half' or 'pairs', not {layout!r}")
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k are both None")
    if first.dim() != 4:
        raise ValueError(f"q and k are [batch, seqlen, heads, headdim], not {tuple(first.shape)}")
    b, L, _, dim = first.shape
    p = _Plan()
    p.dev, p.desc, p.ws = _device(first, q, k, freq, positions, q_out, k_out), abi.RopeDesc(), 0
    d = p.desc
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
    p.likes = [None, None]
    for i, (name, x, y) in enumerate((("q", q, q_out), ("k", k, k_out))):
        if x is None:
            if y is not None:
                raise ValueError(f"an output without its input: {name}")
            continue
        p.likes[i] = _like(x.shape, x.dtype, p.dev)
        _want(x, name, (b, L, x.shape[2] if x.dim() == 4 else -1, dim), first.dtype)
        if y is not None:
            _want(y, name + "_out", x.shape, x.dtype)
        setattr(d, "nheads_" + name, x.shape[2])
        getattr(d, "stride_" + name)[:] = x.stride()[:3]
        getattr(d, f"stride_{name}_out")[:] = (_dense_strides(x.shape) if y is None else y.stride())[:3]
    return p


def _rope(p, st, inverse, q, k, freq, positions, q_out, k_out):
    if q_out is None and q is not None:
        q_out = _new(p.likes[0])
    if k_out is None and k is not None:
        k_out = _new(p.likes[1])
    call = p.lib.ssm_rope_bwd if inverse else p.lib.ssm_rope_fwd
    rc = call(p.desc, _ptr(q), _ptr(k), freq.data_ptr(), _ptr(positions), _ptr(q_out), _ptr(k_out), st)
    if rc:
        abi._check(rc, "ssm_rope_bwd" if inverse else "ssm_rope_fwd")
    return q_out, k_out


def rope(q, k, freq, positions=None, layout="half", magnitude=1.0, q_out=None, k_out=None,
         stream=None):
    """(q, k) with rotary positions on the first ``2 * len(freq)`` values of each head.

    q, k: [batch, seqlen, heads, headdim] (either may be None); ``freq`` from
    :func:`rope_frequencies`; ``positions``: int64 [batch, seqlen] or [seqlen] (default 0, 1, ...);
    ``layout``: "half" pairs value i with i + rot / 2, "pairs" neighbours; ``q_out`` may be ``q`` itself
    and ``k_out`` ``k``, and lie over nothing else of the call."""
    magnitude = float(magnitude)
    p = _plan(("rope", _sig(q), _sig(k), _sig(freq), _sig(positions), layout, magnitude, _sig(q_out), _sig(k_out)),
              _rope_plan, q, k, freq, positions, layout, magnitude, q_out, k_out)
    return _on_device(_rope, p, stream, False, q, k, freq, positions, q_out, k_out)


def rope_backward(dq, dk, freq, positions=None, layout="half", magnitude=1.0, dq_out=None,
                  dk_out=None, stream=None):
    """Gradients of :func:`rope`'s inputs for those of its outputs."""
    magnitude = float(magnitude)
    p = _plan(("rope", _sig(dq), _sig(dk), _sig(freq), _sig(positions), layout, magnitude, _sig(dq_out), _sig(dk_out)),
              _rope_plan, dq, dk, freq, positions, layout, magnitude, dq_out, dk_out)
    return _on_device(_rope, p, stream, True, dq, dk, freq, positions, dq_out, dk_out)


# ---- linear attention ------------------------------------------------------------------

def _la_plan(which, q, k, v, log_decay, lengths, scale, route, states, more):
    """``states``: (name, tensor or None); ``more``: (stride field, tensor or None for a dense
    one, shape)."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are [batch, seqlen, heads, headdim]")
    b, L, h, dk = q.shape
    g, dv = k.shape[2], v.shape[3]
    p = _Plan()
    p.dev = _device(q, k, v, log_decay, lengths, *(t for _, t in states), *(t for _, t, _ in more))
    size = (b, h, dk, dv)
    _want(q, "q", q.shape, q.dtype)
    _want(k, "k", (b, L, g, dk), q.dtype)
    _want(v, "v", (b, L, g, dv), q.dtype)
    _want(log_decay, "log_decay", (h,), torch.float32, True)
    if lengths is not None:
        _want(lengths, "lengths", (b,), torch.int32, True)
    for name, t in states:
        if t is not None:
            _want(t, name, size, torch.float32, True)
    d = p.desc = abi.LinattnDesc()
    d.batch, d.seqlen, d.nheads, d.nheads_kv, d.dim_k, d.dim_v = b, L, h, g, dk, dv
    d.scale, d.dtype_io, d.route = max(dk, 1) ** -0.5 if scale is None else scale, _io(q, "q"), route
    d.stride_q[:], d.stride_k[:], d.stride_v[:] = q.stride()[:3], k.stride()[:3], v.stride()[:3]
    for name, t, shape in more:
        if t is not None:
            _want(t, name, shape, q.dtype)
        getattr(d, "stride_" + name)[:] = (_dense_strides(shape) if t is None else t.stride())[:3]
    p.ws = 0 if which is None else abi.ssm_linattn_workspace_size(d, which)
    p.likes = (_like((b, L, h, dv), q.dtype, p.dev), _like(size, torch.float32, p.dev),
               *(_like(x.shape, q.dtype, p.dev) for x in (q, k, v)))
    return p


def _la_fwd_plan(q, k, v, log_decay, scale, state, lengths, out, state_out, route):
    return _la_plan(abi.PASS_FWD, q, k, v, log_decay, lengths, scale, route,
                    (("state", state), ("state_out", state_out)), (("o", out, (*q.shape[:3], v.shape[-1])),))


def _la_fwd(p, st, q, k, v, log_decay, state, lengths, out, want_state, state_out, workspace):
    if out is None:
        out = _rows_of(p.likes[0], lengths)
    if state_out is None and want_state:
        state_out = _new(p.likes[1])
    ws, n, keep = _workspace(p, workspace)
    rc = p.lib.ssm_linattn_fwd(p.desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                               _ptr(state), _ptr(lengths), out.data_ptr(), _ptr(state_out), ws, n, st)
    if rc:
        abi._check(rc, "ssm_linattn_fwd")
    return out, state_out


def linattn(q, k, v, log_decay, scale=None, state=None, lengths=None, out=None, want_state=True,
            state_out=None, route=abi.LINATTN_AUTO, workspace=None, stream=None):
    """(o, state): linear attention with the decay e^log_decay[h] a head, over whole sequences.

    q [B, L, H, dim_k], k [B, L, G, dim_k], v [B, L, G, dim_v] with H a multiple of G;
    ``scale`` defaults to dim_k ** -0.5; ``state`` fp32 [B, H, dim_k, dim_v] enters (default
    zero).  bf16 outputs of sequences longer than 2048 / max(dim_k, dim_v) are 2.3e-3 from exact
    values in the 2-norm (scores and the state that is read are rounded to bf16), by
    ``route=abi.LINATTN_RECURRENT`` 1.7e-3 in many times the time; states keep 24 bits.

    ``out`` may not lie over q, k or v; ``lengths`` int32 [B]: rows behind them count for nothing and are not written (a given
    ``out`` keeps them, a new one has zeros there).  ``state_out`` takes the final state (may be
    ``state``)."""
    scale = None if scale is None else float(scale)
    p = _plan(("la", _sig(q), _sig(k), _sig(v), _sig(log_decay), scale, _sig(state), _sig(lengths), _sig(out),
               _sig(state_out), route),
              _la_fwd_plan, q, k, v, log_decay, scale, state, lengths, out, state_out, route)
    return _on_device(_la_fwd, p, stream, q, k, v, log_decay, state, lengths, out, want_state, state_out, workspace)


def _la_bwd_plan(q, k, v, log_decay, do, scale, state, dstate, lengths, dq, dk, dv, route):
    return _la_plan(abi.PASS_BWD, q, k, v, log_decay, lengths, scale, route, (("state", state), ("dstate", dstate)),
                    (("o", do, (*q.shape[:3], v.shape[-1])), ("dq", dq, q.shape), ("dk", dk, k.shape),
                     ("dv", dv, v.shape)))


def _la_bwd(p, st, q, k, v, log_decay, do, state, dstate, lengths, dq, dk, dv, workspace):
    if dq is None:
        dq = _rows_of(p.likes[2], lengths)
    if dk is None:
        dk = _rows_of(p.likes[3], lengths)
    if dv is None:
        dv = _rows_of(p.likes[4], lengths)
    din = _new(p.likes[1])
    ws, n, keep = _workspace(p, workspace)
    rc = p.lib.ssm_linattn_bwd(p.desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                               _ptr(state), _ptr(lengths), do.data_ptr(), _ptr(dstate), dq.data_ptr(),
                               dk.data_ptr(), dv.data_ptr(), din.data_ptr(), ws, n, st)
    if rc:
        abi._check(rc, "ssm_linattn_bwd")
    return dq, dk, dv, din


def linattn_backward(q, k, v, log_decay, do, scale=None, state=None, dstate=None, lengths=None,
                     out=None, route=abi.LINATTN_AUTO, workspace=None, stream=None):
    """(dq, dk, dv, dstate): gradients of :func:`linattn` for ``do`` and ``dstate``, that of the
    final state (default zero); the returned dstate is that of the entering ``state``.  As exact
    as :func:`linattn`, by either route.
    ``out``: buffers (dq, dk, dv; each may be None) that lie over no input, whose rows behind ``lengths`` stay as they
    are; new ones have zeros there, so that a sum over a padded batch needs no mask."""
    dq, dk, dv = out if out is not None else (None, None, None)
    scale = None if scale is None else float(scale)
    p = _plan(("la'", _sig(q), _sig(k), _sig(v), _sig(log_decay), _sig(do), scale, _sig(state), _sig(dstate),
               _sig(lengths), _sig(dq), _sig(dk), _sig(dv), route),
              _la_bwd_plan, q, k, v, log_decay, do, scale, state, dstate, lengths, dq, dk, dv, route)
    return _on_device(_la_bwd, p, stream, q, k, v, log_decay, do, state, dstate, lengths, dq, dk, dv, workspace)


def _la_step_plan(q, k, v, log_decay, state, scale, out):
    return _la_plan(None, q, k, v, log_decay, None, scale, abi.LINATTN_AUTO, (("state", state),),
                    (("o", out, (*q.shape[:3], v.shape[-1])),))


def _la_step(p, st, q, k, v, log_decay, state, out):
    if out is None:
        out = _new(p.likes[0])
    rc = p.lib.ssm_linattn_step(p.desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                state.data_ptr(), out.data_ptr(), st)
    if rc:
        abi._check(rc, "ssm_linattn_step")
    return out


def linattn_step(q, k, v, log_decay, state, scale=None, out=None, stream=None):
    """o [B, 1, H, dim_v] of one token (seqlen 1); ``state`` is updated in place; ``out`` may not lie
    over q, k or v."""
    scale = None if scale is None else float(scale)
    p = _plan(("la1", _sig(q), _sig(k), _sig(v), _sig(log_decay), _sig(state), scale, _sig(out)),
              _la_step_plan, q, k, v, log_decay, state, scale, out)
    return _on_device(_la_step, p, stream, q, k, v, log_decay, state, out)
