"""64-bit forms of the layer operators for the tests: the definitions, written with numpy."""
import numpy as np

# half a step of a rounding to the type, relative to the value
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -4}
U32 = 2.0 ** -24


def norm(x, res, w, eps, round_io):
    """(r, y, rstd) with r = round_io(x + res)."""
    r = x if res is None else round_io(x + res)
    rstd = 1.0 / np.sqrt((r * r).mean(-1) + eps)
    y = r * rstd[..., None]
    return r, y if w is None else y * w, rstd


def norm_bwd(dy, r, w, rstd, dr):
    xhat = r * rstd[..., None]
    g = dy if w is None else dy * w
    dx = rstd[..., None] * (g - xhat * (g * xhat).mean(-1, keepdims=True))
    flat = (-1, r.shape[-1])
    return dx if dr is None else dx + dr, (dy * xhat).reshape(flat).sum(0)


def rope(x, freq, pos, layout, magnitude=1.0, sign=1.0):
    """x [B, L, H, D]; pos [B, L]."""
    m = 2 * len(freq)
    ang = np.asarray(pos, dtype=np.float64)[..., None, None] * freq
    c, s = magnitude * np.cos(ang), sign * magnitude * np.sin(ang)
    a, b = (np.s_[..., : m // 2], np.s_[..., m // 2: m]) if layout == "half" else (np.s_[..., 0:m:2], np.s_[..., 1:m:2])
    y = x.copy()
    y[a], y[b] = x[a] * c - x[b] * s, x[a] * s + x[b] * c
    return y


def _rep(x, h):
    return np.repeat(x, h // x.shape[2], axis=2)


def linattn(q, k, v, g, scale, s0=None, lengths=None):
    """(o, state): o is 0 behind the lengths."""
    B, L, H, dk = q.shape
    k, v = _rep(k, H), _rep(v, H)
    dv = v.shape[3]
    lam = np.exp(g)[None, :, None, None]
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    S = np.zeros((B, H, dk, dv)) if s0 is None else s0.copy()
    o = np.zeros((B, L, H, dv))
    for t in range(L):
        on = t < n
        S[on] = (lam * S)[on] + np.einsum("bhk,bhv->bhkv", k[on, t], v[on, t])
        o[on, t] = scale * np.einsum("bhk,bhkv->bhv", q[on, t], S[on])
    return o, S


def linattn_bwd(q, k, v, g, scale, do, s0=None, ds=None, lengths=None):
    """(dq, dk, dv, dstate): 0 behind the lengths."""
    B, L, H, dk = q.shape
    G, dv = k.shape[2], v.shape[3]
    kk, vv = _rep(k, H), _rep(v, H)
    lam = np.exp(g)[None, :, None, None]
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    S = np.zeros((B, H, dk, dv)) if s0 is None else s0.copy()
    dq = np.zeros(q.shape)
    for t in range(L):
        on = t < n
        S[on] = (lam * S)[on] + np.einsum("bhk,bhv->bhkv", kk[on, t], vv[on, t])
        dq[on, t] = scale * np.einsum("bhv,bhkv->bhk", do[on, t], S[on])
    A = np.zeros((B, H, dk, dv)) if ds is None else ds.copy()
    dkk, dvv = np.zeros(kk.shape), np.zeros(vv.shape)
    for t in reversed(range(L)):
        on = t < n
        A[on] += scale * np.einsum("bhk,bhv->bhkv", q[on, t], do[on, t])
        dkk[on, t] = np.einsum("bhv,bhkv->bhk", vv[on, t], A[on])
        dvv[on, t] = np.einsum("bhk,bhkv->bhv", kk[on, t], A[on])
        A[on] = (lam * A)[on]
    return dq, dkk.reshape(B, L, G, H // G, dk).sum(3), dvv.reshape(B, L, G, H // G, dv).sum(3), A
