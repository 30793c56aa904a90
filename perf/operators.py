"""The language-model operators around the scan, as measured: cases, inputs, plain forms and 64-bit values.

Three operators, the parts of one layer whose mixer is linear attention:

* ``norm``: residual addition, root-mean-square norm, output in the I/O type or in
  8 bits (e4m3) with a scale a row or a block of 128 columns; with its gradient.
* ``rope``: rotary positions on queries and keys, interleaved or half layout, all or
  part of the head, given frequencies (scaled ones for long contexts); with its gradient.
* ``linattn``: linear attention with a decay a head,
  S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale q_t S_t, over whole prompts (``prompt``),
  with its gradient (``train``) and one token at a time (``step``).

``run`` computes them with elementary torch operations in 32 bits, or, where ``own``
is set, with this package's entry points.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
CHUNK = 128          # of the plain form of the linear attention
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token each of 8 sequences: the latency of a decoding step's positions
        {"name": "rope decode 8x1", "op": "rope", "train": False, "batch": 8, "seqlen": 1, "heads": 16,
         "kv": 4, "dim": 128, "rot": 128, "layout": "half", "offset": 70001, "dtype": "bf16"},
        # a batch of prompts, interleaved pairs on half of each head (heads of the Mamba-2 workload)
        {"name": "rope prompt 4x2048", "op": "rope", "train": False, "batch": 4, "seqlen": 2048, "heads": 24,
         "kv": 3, "dim": 64, "rot": 32, "layout": "pairs", "offset": 0, "dtype": "bf16"},
        # a training step over long sequences: the rotation and the gradient through it
        {"name": "rope train 4x16384", "op": "rope", "train": True, "batch": 4, "seqlen": 16384, "heads": 16,
         "kv": 16, "dim": 128, "rot": 128, "layout": "half", "offset": 0, "dtype": "bf16"},
        # a decoding step's norm in front of an 8-bit projection
        {"name": "norm decode 8x2048 e4m3", "op": "norm", "train": False, "rows": 8, "dim": 2048,
         "residual": True, "quant": "block", "dtype": "bf16"},
        # the norm over the rows of the HybridMamba workload (8 x 8192 tokens, 32 heads of 64)
        {"name": "norm prompt 65536x2048 e4m3", "op": "norm", "train": False, "rows": 65536, "dim": 2048,
         "residual": True, "quant": "row", "dtype": "bf16"},
        # a training step's norm, an odd number of rows, heads of the Mamba-2 workload (24 of 64)
        {"name": "norm train 8191x1536", "op": "norm", "train": True, "rows": 8191, "dim": 1536,
         "residual": True, "quant": "none", "dtype": "bf16"},
        # decoding: one token of 64 sequences, the state read and written in place
        {"name": "linattn step 64", "op": "step", "batch": 64, "heads": 16, "kv": 16, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # one short prompt of an odd length
        {"name": "linattn prompt 1x257", "op": "prompt", "batch": 1, "seqlen": 257, "heads": 16, "kv": 16,
         "dk": 64, "dv": 64, "ragged": False, "dtype": "bf16"},
        # prompts of different lengths in one padded batch, shared key and value heads
        {"name": "linattn prompt 4x2048 ragged", "op": "prompt", "batch": 4, "seqlen": 2048, "heads": 24,
         "kv": 3, "dk": 128, "dv": 64, "ragged": True, "dtype": "bf16"},
        # the long prompts of the SSD-MIMO workload's batch
        {"name": "linattn prompt 4x16384", "op": "prompt", "batch": 4, "seqlen": 16384, "heads": 16, "kv": 16,
         "dk": 128, "dv": 128, "ragged": False, "dtype": "bf16"},
        # a training step with grouped heads: outputs and every gradient
        {"name": "linattn train 4x4096", "op": "train", "batch": 4, "seqlen": 4096, "heads": 16, "kv": 4,
         "dk": 128, "dv": 128, "ragged": False, "dtype": "bf16"},
        # small heads in 32 bits, as the tiny hybrid workload has them
        {"name": "linattn train fp32 2x300", "op": "train", "batch": 2, "seqlen": 300, "heads": 4, "kv": 2,
         "dk": 16, "dv": 24, "ragged": False, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; none costs more than the largest listed one of its operator."""
    while True:
        op = rng.choice(["rope", "norm", "step", "prompt", "prompt", "train", "train"])
        dtype = "bf16" if rng.random() < 0.8 else "fp32"
        if op == "norm":
            train = rng.random() < 0.5
            c = {"op": op, "train": train, "rows": _log(rng, 1, 65536), "dim": 8 * _log(rng, 8, 1024),
                 "residual": rng.random() < 0.7, "quant": "none" if train else rng.choice(["none", "row", "block"]),
                 "dtype": dtype}
            if c["quant"] == "block":
                c["dim"] = 128 * max(1, c["dim"] // 128)
            if rng.random() < 0.2 and c["quant"] == "none":
                c["dim"] += rng.randrange(1, 8)
            if c["rows"] * c["dim"] > 65536 * 2048:
                continue
            return c
        if op == "rope":
            dim = rng.choice([32, 64, 80, 96, 128, 256])
            kv = rng.choice([1, 2, 4, 8])
            c = {"op": op, "train": rng.random() < 0.5, "batch": _log(rng, 1, 64), "seqlen": _log(rng, 1, 16384),
                 "heads": kv * rng.choice([1, 2, 3, 4, 8]), "kv": kv, "dim": dim,
                 "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "layout": rng.choice(["half", "pairs"]),
                 "offset": rng.choice([0, 0, _log(rng, 1, 1 << 20)]), "dtype": dtype}
            if c["batch"] * c["seqlen"] * (c["heads"] + kv) * dim > 4 * 16384 * 32 * 128:
                continue
            return c
        kv = rng.choice([1, 2, 3, 4, 8, 16])
        c = {"op": op, "batch": _log(rng, 1, 128 if op == "step" else 8), "heads": kv * rng.choice([1, 1, 2, 4, 8]), "kv": kv,
             "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]), "dtype": dtype}
        if dtype == "fp32" or rng.random() < 0.1:
            c["dk"], c["dv"] = rng.randrange(8, 129), rng.randrange(8, 129)
        if op == "step":
            if c["batch"] * c["heads"] > 64 * 32:
                continue
            return c
        general = dtype == "fp32" or c["dk"] % 64 or c["dv"] % 64
        c |= {"seqlen": _log(rng, 1, 2048 if general else 16384), "ragged": rng.random() < 0.3}
        most = 4 * 2048 * 8 if general else 4 * 16384 * 16 if op == "prompt" else 4 * 4096 * 16
        if c["batch"] * c["seqlen"] * c["heads"] > most:
            continue
        return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    return x.mul_(scale).to(dtype)


def _frequencies(rot):
    """Radians a position of each pair (base 10000, positions interpolated by 4 as after a context extension)."""
    return 10000.0 ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot) / 4.0


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": dict(c)}
    if c["op"] == "norm":
        n, d = c["rows"], c["dim"]
        s["x"] = _normal(g, (n, d), dt)
        s["residual"] = _normal(g, (n, d), dt, 2.0) if c["residual"] else None
        s["weight"] = _normal(g, (d,), torch.float32, 0.2) + 1.0
        if c["train"]:
            s["dy"], s["dr"] = _normal(g, (n, d), dt), _normal(g, (n, d), dt) if c["residual"] else None
        return s
    b, h, kv = c["batch"], c["heads"], c["kv"]
    if c["op"] == "rope":
        L, d = c["seqlen"], c["dim"]
        s["q"], s["k"] = _normal(g, (b, L, h, d), dt), _normal(g, (b, L, kv, d), dt)
        start = torch.randint(0, 64, (b, 1), generator=g, device="cuda") + c["offset"]
        s["positions"] = start + torch.arange(L, device="cuda")[None, :]
        s["freq"] = torch.from_numpy(_frequencies(c["rot"])).cuda()
        if c["train"]:
            s["dq"], s["dk"] = _normal(g, (b, L, h, d), dt), _normal(g, (b, L, kv, d), dt)
        return s
    dk, dv = c["dk"], c["dv"]
    L = c.get("seqlen", 1)
    s["q"], s["k"] = _normal(g, (b, L, h, dk), dt), _normal(g, (b, L, kv, dk), dt)
    s["v"] = _normal(g, (b, L, kv, dv), dt)
    # decays of retention: memories from about one token to a thousand
    u = torch.empty(h, dtype=torch.float32, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g)
    s["log_decay"] = -u.exp()
    s["scale"] = dk ** -0.5
    s["state"] = _normal(g, (b, h, dk, dv), torch.float32)
    if c["op"] == "step":
        return s
    s["lengths"] = None
    if c["ragged"]:
        s["lengths"] = torch.randint(0, L + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        s["lengths"][0] = L
    # a caller's output buffers; rows behind a sequence's length stay as they are
    s["o"] = torch.zeros((b, L, h, dv), dtype=dt, device="cuda")
    if c["op"] == "train":
        s["do"] = _normal(g, (b, L, h, dv), dt)
        s["dstate"] = _normal(g, (b, h, dk, dv), torch.float32)
        s["grads"] = [torch.zeros_like(s[x]) for x in ("q", "k", "v")]
    return s


# ---- plain forms ------------------------------------------------------------------

def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    r = s["x"].float()
    if s["residual"] is not None:
        r = (r + s["residual"].float()).to(dt).float()
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-5)
    y = r * rstd * s["weight"]
    out = {}
    if s["residual"] is not None:
        out["r"] = r.to(dt)
    if c["quant"] == "none":
        out["y"] = y.to(dt)
    else:
        blocks = y.unflatten(-1, (-1, 128 if c["quant"] == "block" else c["dim"]))
        top = blocks.abs().amax(-1, keepdim=True)
        out["scales"] = (top / E4M3_MAX).squeeze(-1)
        out["y8"] = (blocks * (E4M3_MAX / top)).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2).to(torch.float8_e4m3fn)
    if c["train"]:
        xhat, dy = r * rstd, s["dy"].float()
        wdy = dy * s["weight"]
        dx = rstd * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True))
        if s["dr"] is not None:
            dx = dx + s["dr"].float()
        out["dx"] = dx.to(dt)
        out["dweight"] = (dy * xhat).sum(0)
    return out


def _rotate(x, cos, sin, rot, layout):
    head, rest = x[..., :rot].to(cos.dtype), x[..., rot:]
    if layout == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), rest], -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[..., None, None] * s["freq"]   # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    out = [_rotate(s[x], cos, sin, c["rot"], c["layout"]) for x in ("q", "k")]
    if c["train"]:
        out += [_rotate(s[x], cos, -sin, c["rot"], c["layout"]) for x in ("dq", "dk")]
    return out


def _decayed(q, k, v, g):
    """sum_{s <= t} e^{g (t - s)} (q_t . k_s) v_s for [B, H, L, d] inputs, chunk by chunk."""
    L = q.shape[2]
    n = -(-L // CHUNK)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - L)).unflatten(2, (n, CHUNK)) for x in (q, k, v))
    i = torch.arange(CHUNK, device=q.device, dtype=torch.float32)
    c = torch.arange(n, device=q.device, dtype=torch.float32)
    g = g[:, None, None]
    w = torch.where(i[:, None] >= i[None, :], torch.exp(g * (i[:, None] - i[None, :]).clamp(min=0)), 0.0)
    o = ((q @ k.transpose(-1, -2)) * w[:, None]) @ v
    if n > 1:
        local = (k * torch.exp(g * (CHUNK - 1 - i)[None, :, None])[:, None]).transpose(-1, -2) @ v
        far = (c[:, None] - 1 - c[None, :]) * CHUNK
        carry = torch.where(far >= 0, torch.exp(g * far.clamp(min=0)), 0.0)
        entering = (carry @ local.flatten(-2)).unflatten(-1, local.shape[-2:])
        o = o + (q * torch.exp(g * (i + 1)[None, :, None])[:, None]) @ entering
    return o.flatten(2, 3)[:, :, :L]


def _heads(x, h, valid):
    """[B, L, G, d] in 32 bits as [B, H, L, d], key and value heads repeated, nothing behind the lengths."""
    x = torch.where(valid[:, :, None, None], x.float(), 0.0).transpose(1, 2)
    return x.repeat_interleave(h // x.shape[1], dim=1)


def _plain_linattn(s):
    c, dt, g, scale = s["case"], s["q"].dtype, s["log_decay"], s["scale"]
    b, L, h, _ = s["q"].shape
    t = torch.arange(L, device="cuda", dtype=torch.float32)
    length = s["lengths"].float() if s["lengths"] is not None else torch.full((b,), float(L), device="cuda")
    valid = t[None, :] < length[:, None]
    q, k, v = (_heads(s[x], h, valid) for x in ("q", "k", "v"))
    gh = g[None, :, None]
    since = torch.exp(gh * (t + 1)[None, None, :])[..., None]                                        # e^{g (t + 1)}
    until = torch.exp(gh * (length[:, None, None] - 1 - t[None, None, :]).clamp(min=0))[..., None]   # e^{g (T - 1 - t)}
    whole = torch.exp(gh[..., None] * length[:, None, None, None])
    o = scale * (_decayed(q, k, v, g) + (q * since) @ s["state"])
    keep = valid[:, :, None, None]
    out = {"o": torch.where(keep, o.transpose(1, 2).to(dt), s["o"]),
           "state": whole * s["state"] + (k * until).transpose(-1, -2) @ v}
    if c["op"] == "train":
        do = _heads(s["do"], h, valid)
        dq = scale * (_decayed(do, v, k, g) + (do * since) @ s["state"].transpose(-1, -2))
        rq, rk, rv, rdo = (x.flip(2) for x in (q, k, v, do))
        dk = scale * _decayed(rv, rdo, rq, g).flip(2) + (v * until) @ s["dstate"].transpose(-1, -2)
        dv = scale * _decayed(rk, rq, rdo, g).flip(2) + (k * until) @ s["dstate"]
        group = lambda x: x.unflatten(1, (c["kv"], -1)).sum(2)  # noqa: E731
        grads = [x.transpose(1, 2).to(dt) for x in (dq, group(dk), group(dv))]
        out["dq"], out["dk"], out["dv"] = (torch.where(keep, x, y) for x, y in zip(grads, s["grads"]))
        out["dstate"] = whole * s["dstate"] + scale * ((q * since).transpose(-1, -2) @ do)
    return out


def _plain_step(s):
    h = s["q"].shape[2]
    q, k, v = s["q"][:, 0].float(), s["k"][:, 0].float(), s["v"][:, 0].float()
    k, v = k.repeat_interleave(h // k.shape[1], 1), v.repeat_interleave(h // v.shape[1], 1)
    s["state"].mul_(s["log_decay"].exp()[None, :, None, None]).add_(k[..., None] * v[..., None, :])
    o = s["scale"] * (q[..., None, :] @ s["state"]).squeeze(-2)
    return {"o": o.to(s["q"].dtype)[:, None], "state": s["state"]}


# ---- the framework's calls -----------------------------------------------------------

def _own_norm(s):
    from selective_diagonal_state_b200 import layer
    c = s["case"]
    f = layer.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=1e-5,
                      quant=None if c["quant"] == "none" else c["quant"], want_rstd=c["train"])
    out = {}
    if s["residual"] is not None:
        out["r"] = f.r
    if c["quant"] == "none":
        out["y"] = f.y
    else:
        out["scales"], out["y8"] = f.scales, f.y8
    if c["train"]:
        out["dx"], out["dweight"] = layer.rmsnorm_backward(s["dy"], f.r, s["weight"], f.rstd, dr=s["dr"])
    return out


def _own_rope(s):
    from selective_diagonal_state_b200 import layer
    c = s["case"]
    out = list(layer.rope(s["q"], s["k"], s["freq"], s["positions"], layout=c["layout"]))
    if c["train"]:
        out += layer.rope_backward(s["dq"], s["dk"], s["freq"], s["positions"], layout=c["layout"])
    return out


def _own_linattn(s):
    from selective_diagonal_state_b200 import layer
    o, state = layer.linattn(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], state=s["state"],
                             lengths=s["lengths"], out=s["o"])
    out = {"o": o, "state": state}
    if s["case"]["op"] == "train":
        out["dq"], out["dk"], out["dv"], out["dstate"] = layer.linattn_backward(
            s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"], state=s["state"],
            dstate=s["dstate"], lengths=s["lengths"], out=s["grads"])
    return out


def _own_step(s):
    from selective_diagonal_state_b200 import layer
    o = layer.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
    return {"o": o, "state": s["state"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_norm if op == "norm" else _own_rope if op == "rope" else _own_step if op == "step" else _own_linattn)(state)
    return (_plain_norm if op == "norm" else _plain_rope if op == "rope" else _plain_step if op == "step" else _plain_linattn)(state)


def work(case):
    """Every input read once and every output written once; the products of the recurrence, token by token."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["rows"] * c["dim"]
        by = n * e * (3 if c["residual"] else 1)
        by += n * e if c["quant"] == "none" else n + 4 * c["rows"] * (c["dim"] // 128 if c["quant"] == "block" else 1)
        fl = 6 * n
        if c["train"]:
            by += n * e * (3 if c["residual"] else 2) + (4 + 4) * c["dim"]
            fl += 12 * n
        return {"bytes": by + 4 * c["dim"], "flops": fl}
    if c["op"] == "rope":
        n = c["batch"] * c["seqlen"] * (c["heads"] + c["kv"]) * c["dim"]
        k = 2 if c["train"] else 1
        return {"bytes": k * 2 * n * e + 8 * c["batch"] * c["seqlen"], "flops": k * 3 * n * c["rot"] / c["dim"]}
    h, kv, dk, dv = c["heads"], c["kv"], c["dk"], c["dv"]
    tok = c["batch"] * c.get("seqlen", 1)
    st = 4 * c["batch"] * h * dk * dv
    by = tok * e * (h * (dk + dv) + kv * (dk + dv)) + 2 * st
    fl = 5.0 * tok * h * dk * dv
    if c["op"] == "train":   # q, k, v stay: the upstream gradients come in, four gradients go out
        by += tok * e * (h * dv + h * dk + kv * (dk + dv)) + 2 * st
        fl *= 3
    return {"bytes": by, "flops": fl}


# ---- 64-bit values from the definitions ------------------------------------------------

def _exact_norm(s):
    c = s["case"]
    r = s["x"].double()
    if s["residual"] is not None:
        r = (s["x"] + s["residual"]).double()     # one rounding: the stored sum is what is normalised
    d = c["dim"]
    inv = 1.0 / torch.sqrt((r * r).sum(-1, keepdim=True) / d + 1e-5)
    w = s["weight"].double()
    y = r * inv * w
    out = {}
    if s["residual"] is not None:
        out["r"] = r
    if c["quant"] == "none":
        out["y"] = y
    else:
        width = 128 if c["quant"] == "block" else d
        top = y.abs().reshape(c["rows"], d // width, width).max(-1).values
        out["scales"] = top / E4M3_MAX
        out["y8"] = y / out["scales"].repeat_interleave(width, -1)
    if c["train"]:
        # J^T (w dy) with J = d(r inv)/dr
        up = s["dy"].double() * w
        dot = (up * r).sum(-1, keepdim=True)
        out["dx"] = inv * up - r * inv ** 3 * dot / d
        if s["dr"] is not None:
            out["dx"] += s["dr"].double()
        out["dweight"] = (s["dy"].double() * r * inv).sum(0)
    return out


def _exact_rope(s):
    c = s["case"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, :, None, None] * s["freq"])

    def spin(x, z):
        x, m = x.double().clone(), c["rot"]
        a, b = (slice(0, m // 2), slice(m // 2, m)) if c["layout"] == "half" else (slice(0, m, 2), slice(1, m, 2))
        y = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * z
        x[..., a], x[..., b] = y.real, y.imag
        return x

    out = [spin(s["q"], turn), spin(s["k"], turn)]
    if c["train"]:
        out += [spin(s["dq"], turn.conj()), spin(s["dk"], turn.conj())]
    return out


def _exact_linattn(s):
    """The recurrence one token after the other, and the adjoint recurrence backwards."""
    c = s["case"]
    b, L, h, dk = s["q"].shape
    rep, train = h // c["kv"], c["op"] == "train"
    lam = s["log_decay"].double().exp()[None, :, None, None]
    n = s.get("lengths")
    n = torch.full((b,), L, device="cuda") if n is None else n
    scale = s["scale"]

    def at(x, t):
        x = x[:, t].double()
        return x if x.shape[1] == h else x.repeat_interleave(rep, 1)

    S = s["state"].double().clone()
    o = torch.zeros((b, L, h, c["dv"]), dtype=torch.float64, device="cuda")
    dq = torch.zeros((b, L, h, dk), dtype=torch.float64, device="cuda") if train else None
    for t in range(L):
        on = (t < n)[:, None, None, None]
        new = torch.addcmul(lam * S, at(s["k"], t)[..., None], at(s["v"], t)[..., None, :])
        S = torch.where(on, new, S) if c.get("ragged") else new
        o[:, t] = scale * torch.einsum("bhk,bhkv->bhv", at(s["q"], t), S)
        if train:
            dq[:, t] = scale * torch.einsum("bhv,bhkv->bhk", at(s["do"], t), S)
    live = (torch.arange(L, device="cuda")[None] < n[:, None])[..., None, None]
    out = {"o": torch.where(live, o, 0.0), "state": S}
    if not train:
        return out
    G = s["dstate"].double().clone()
    dk_, dv_ = torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
    for t in reversed(range(L)):
        on = (t < n)[:, None, None, None]
        A = torch.addcmul(G, scale * at(s["q"], t)[..., None], at(s["do"], t)[..., None, :])   # dL/dS_t
        dk_[:, t] = torch.einsum("bhv,bhkv->bhk", at(s["v"], t), A).unflatten(1, (c["kv"], rep)).sum(2)
        dv_[:, t] = torch.einsum("bhk,bhkv->bhv", at(s["k"], t), A).unflatten(1, (c["kv"], rep)).sum(2)
        G = torch.where(on, lam * A, G) if c["ragged"] else lam * A
    out |= {"dq": torch.where(live, dq, 0.0), "dk": torch.where(live, dk_, 0.0), "dv": torch.where(live, dv_, 0.0),
            "dstate": G}
    return out


def exact(case, seed):
    s = prepare(case, seed)
    out = (_exact_norm if case["op"] == "norm" else _exact_rope if case["op"] == "rope" else _exact_linattn)(s)
    if case["op"] == "step":
        out = {"o": out["o"], "state": out["state"]}
    return out
