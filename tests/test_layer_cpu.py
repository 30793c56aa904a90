"""The layer operators' host side: descriptors, refusals before any launch, rotary
frequencies, and the 64-bit gradients against differences."""
import ctypes
import math

import numpy as np
import pytest

from selective_diagonal_state_b200 import abi, build
from tests import layer_ref as R

FAKE = 1 << 40  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load_library()


def err(lib):
    return lib.ssm_scan_last_error().decode()


def norm_desc(rows=4, dim=256, **kw):
    d = abi.RmsnormDesc(rows=rows, dim=dim, eps=1e-5, dtype_io=abi.DTYPE_BF16)
    for s in ("x", "residual", "r", "y", "y8", "dy", "dr", "dx"):
        setattr(d, "stride_" + s, dim)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def rope_desc(batch=2, seqlen=8, hq=4, hk=2, dim=64, rot=64, **kw):
    d = abi.RopeDesc(batch=batch, seqlen=seqlen, nheads_q=hq, nheads_k=hk, headdim=dim, rot_dim=rot,
                     magnitude=1.0, dtype_io=abi.DTYPE_BF16)
    for s, h in (("q", hq), ("k", hk), ("q_out", hq), ("k_out", hk)):
        getattr(d, "stride_" + s)[:] = (seqlen * h * dim, h * dim, dim)
    d.stride_pos[:] = (seqlen, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def la_desc(batch=2, seqlen=8, h=4, g=2, dk=64, dv=64, **kw):
    d = abi.LinattnDesc(batch=batch, seqlen=seqlen, nheads=h, nheads_kv=g, dim_k=dk, dim_v=dv,
                        scale=1.0, dtype_io=abi.DTYPE_BF16)
    for s, n, dim in (("q", h, dk), ("k", g, dk), ("v", g, dv), ("o", h, dv), ("dq", h, dk),
                      ("dk", g, dk), ("dv", g, dv)):
        getattr(d, "stride_" + s)[:] = (seqlen * n * dim, n * dim, dim)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_descriptor_sizes(lib):
    """No padding: ten int64 and four 4-byte fields; six int64, 14 strides and four; six
    int64, 21 strides and four."""
    assert ctypes.sizeof(abi.RmsnormDesc) == 10 * 8 + 4 * 4
    assert ctypes.sizeof(abi.RopeDesc) == 6 * 8 + 14 * 8 + 4 * 4
    assert ctypes.sizeof(abi.LinattnDesc) == 6 * 8 + 21 * 8 + 4 * 4


@pytest.mark.parametrize("kw,args,code,word", [
    (dict(rows=-1), {}, -1, "rows"),
    (dict(dim=0), {}, -1, "dim"),
    (dict(eps=-1.0), {}, -1, "eps"),
    (dict(eps=math.nan), {}, -1, "eps"),
    (dict(dtype_io=2), {}, -1, "dtype"),
    (dict(quant=3), {}, -1, "quant"),
    (dict(quant=2, dim=200), {}, -1, "128"),
    (dict(reserved_=1), {}, -1, "reserved"),
    (dict(dim=(1 << 20) + 8), {}, -2, "dim"),
    (dict(stride_x=-1), {}, -1, "negative"),
    (dict(stride_y=0), {}, -1, "overlaps"),
    ({}, dict(x=None), -1, "x"),
    ({}, dict(y=None), -1, "y"),
    ({}, dict(r=None), -1, "r is"),
    ({}, dict(x=FAKE + 1), -3, "aligned"),
    (dict(quant=1), dict(y8=None), -1, "y8"),
    (dict(quant=1), dict(scales=None), -1, "scales"),
])
def test_rmsnorm_refusals(lib, kw, args, code, word):
    a = dict(x=FAKE, res=FAKE, w=FAKE, r=FAKE, y=FAKE, y8=FAKE, scales=FAKE, rstd=FAKE) | args
    rc = lib.ssm_rmsnorm_fwd(norm_desc(**kw), a["x"], a["res"], a["w"], a["r"], a["y"], a["y8"],
                             a["scales"], a["rstd"], None)
    assert rc == code and word in err(lib), (rc, err(lib))


def test_rmsnorm_backward_refusals(lib):
    d = norm_desc()
    need = lib.ssm_rmsnorm_workspace_size(d)
    assert need > 0 and need % 256 == 0
    assert lib.ssm_rmsnorm_bwd(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == -6
    assert lib.ssm_rmsnorm_bwd(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need - 1, None) == -6
    assert lib.ssm_rmsnorm_bwd(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 16, need, None) == -3
    assert lib.ssm_rmsnorm_bwd(d, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, need, None) == -1
    assert "rstd" in err(lib)
    assert lib.ssm_rmsnorm_bwd(norm_desc(stride_dx=8), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, 0, None) == -1
    assert lib.ssm_rmsnorm_workspace_size(norm_desc(rows=0)) == 0
    assert lib.ssm_rmsnorm_fwd(None, *[FAKE] * 8, None) == -1
    assert lib.ssm_rmsnorm_fwd(norm_desc(rows=0), *[None] * 8, None) == 0     # nothing to do


@pytest.mark.parametrize("kw,args,code,word", [
    (dict(batch=-1), {}, -1, "batch"),
    (dict(rot_dim=63), {}, -1, "rot_dim"),
    (dict(rot_dim=66), {}, -1, "rot_dim"),
    (dict(rot_dim=0), {}, -1, "rot_dim"),
    (dict(layout=2), {}, -1, "layout"),
    (dict(magnitude=math.inf), {}, -1, "magnitude"),
    (dict(dtype_io=5), {}, -1, "dtype"),
    (dict(reserved_=2), {}, -1, "reserved"),
    (dict(seqlen=1 << 31), {}, -2, "sizes"),
    ({}, dict(q=None, k=None), -1, "both"),
    ({}, dict(qo=None), -1, "q_out"),
    ({}, dict(freq=None), -1, "freq"),
    ({}, dict(freq=FAKE + 4), -3, "freq"),
    ({}, dict(pos=FAKE + 4), -3, "positions"),
    ({}, dict(k=FAKE + 1), -3, "k is"),
])
def test_rope_refusals(lib, kw, args, code, word):
    a = dict(q=FAKE, k=FAKE, freq=FAKE, pos=FAKE, qo=FAKE, ko=FAKE) | args
    for f in (lib.ssm_rope_fwd, lib.ssm_rope_bwd):
        rc = f(rope_desc(**kw), a["q"], a["k"], a["freq"], a["pos"], a["qo"], a["ko"], None)
        assert rc == code and word in err(lib), (rc, err(lib))


def test_rope_stride_refusals(lib):
    d = rope_desc()
    d.stride_q_out[2] = 0
    assert lib.ssm_rope_fwd(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -1 and "overlaps" in err(lib)
    d = rope_desc()
    d.stride_k_out[1] = d.stride_k_out[2]
    assert lib.ssm_rope_fwd(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -1 and "stride" in err(lib)


def test_rope_frequencies(lib):
    d, base = 64, 10000.0
    i = np.arange(d // 2)
    plain = base ** (-2.0 * i / d)
    np.testing.assert_allclose(abi.ssm_rope_frequencies(d, base), plain, rtol=1e-14)
    np.testing.assert_allclose(abi.ssm_rope_frequencies(d, base, abi.ROPE_LINEAR, 4.0), plain / 4, rtol=1e-14)
    np.testing.assert_allclose(abi.ssm_rope_frequencies(d, base, abi.ROPE_NTK, 8.0),
                               (base * 8.0 ** (d / (d - 2))) ** (-2.0 * i / d), rtol=1e-13)
    got = np.array(abi.ssm_rope_frequencies(d, base, abi.ROPE_BANDS, 8.0, 1.0, 4.0, 8192.0))
    turns = 8192.0 * plain / (2 * math.pi)
    keep = np.clip((turns - 1.0) / 3.0, 0.0, 1.0)
    np.testing.assert_allclose(got, plain * (keep + (1 - keep) / 8.0), rtol=1e-13)
    assert got[0] == plain[0] and got[-1] == pytest.approx(plain[-1] / 8.0)   # fast pairs kept, slow ones divided
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(base=0.0), dict(scaling=4), dict(scaling=1, factor=0.5),
                dict(scaling=2, rot_dim=2), dict(scaling=3, factor=2.0, low_turns=4.0, high_turns=4.0, original_context=8.0),
                dict(scaling=3, factor=2.0, low_turns=1.0, high_turns=4.0)):
        with pytest.raises(abi.SsmError) as e:
            abi.ssm_rope_frequencies(**(dict(rot_dim=64, base=1e4) | bad))
        assert e.value.code == -1


@pytest.mark.parametrize("kw,code,word", [
    (dict(batch=-1), -1, "batch"),
    (dict(nheads_kv=3), -1, "nheads"),
    (dict(nheads=0), -1, "nheads"),
    (dict(dim_k=0), -1, "dim_k"),
    (dict(dim_k=257), -2, "257"),
    (dict(dim_v=300), -2, "300"),
    (dict(route=2), -1, "route"),
    (dict(reserved_=1), -1, "reserved"),
    (dict(dtype_io=2), -1, "dtype"),
    (dict(seqlen=1 << 31), -2, "sizes"),
    (dict(batch=1 << 20), -2, "sizes"),
])
def test_linattn_descriptor_refusals(lib, kw, code, word):
    d = la_desc(**kw)
    assert lib.ssm_linattn_fwd(d, *[FAKE] * 8, None, 0, None) == code and word in err(lib), err(lib)
    assert lib.ssm_linattn_bwd(d, *[FAKE] * 12, None, 0, None) == code
    d1 = la_desc(**(dict(kw) | ({} if "seqlen" in kw else dict(seqlen=1))))
    assert lib.ssm_linattn_step(d1, *[FAKE] * 6, None) == code
    assert lib.ssm_linattn_workspace_size(d, abi.PASS_BWD) == 0


def test_linattn_pointer_refusals(lib):
    d = la_desc()
    names = ["q", "k", "v", "log_decay", "state_in", "lengths", "o", "state_out"]

    def fwd(**kw):
        a = dict.fromkeys(names, FAKE) | kw
        return lib.ssm_linattn_fwd(d, *[a[n] for n in names], None, 0, None)

    for n in ("q", "k", "v", "log_decay"):
        assert fwd(**{n: None}) == -1 and n in err(lib)
    assert fwd(o=None, state_out=None) == -1 and "both" in err(lib)
    for n, off in (("state_in", 2), ("state_out", 2), ("lengths", 2), ("q", 1), ("o", 1)):
        assert fwd(**{n: FAKE + off}) == -3 and n in err(lib)
    bn = ["q", "k", "v", "log_decay", "state_in", "lengths", "do", "dstate_out", "dq", "dk", "dv", "dstate_in"]

    def bwd(ws=None, n=0, **kw):
        a = dict.fromkeys(bn, FAKE) | dict(dstate_in=FAKE + 256) | kw
        return lib.ssm_linattn_bwd(d, *[a[x] for x in bn], ws, n, None)

    for n in ("q", "k", "v", "log_decay", "do", "dq", "dk", "dv"):
        assert bwd(**{n: None}) == -1 and n in err(lib)
    assert bwd(dstate_in=FAKE) == -1 and "dstate" in err(lib)
    need = abi.ssm_linattn_workspace_size(d, abi.PASS_BWD)
    assert need >= 2 * 8 * 4 * (64 + 64) * 4     # dk and dv of every head
    assert bwd() == -6 and str(need) in err(lib)
    assert bwd(FAKE, need - 1) == -6
    assert bwd(FAKE + 16, need) == -3
    assert lib.ssm_linattn_step(d, *[FAKE] * 6, None) == -1 and "one token" in err(lib)
    d1 = la_desc(seqlen=1)
    assert lib.ssm_linattn_step(d1, FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == -1
    assert lib.ssm_linattn_step(d1, FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == -1


def test_linattn_stride_refusals(lib):
    for f in ("stride_o", "stride_dq", "stride_dk", "stride_dv"):
        d = la_desc()
        getattr(d, f)[1] = 0
        rc = (lib.ssm_linattn_fwd(d, *[FAKE] * 8, None, 0, None) if f == "stride_o" else
              lib.ssm_linattn_bwd(d, *[FAKE] * 11, FAKE + 256, None, 0, None))
        assert rc == -1 and "overlaps" in err(lib)
        d = la_desc()
        getattr(d, f)[0] = -4
        assert lib.ssm_linattn_workspace_size(d, abi.PASS_BWD) == 0 and "negative" in err(lib)


def test_outputs_that_overlap_are_refused(lib):
    """Written rows are nested in some order of the dimensions; any order is taken."""
    d = la_desc()       # [2, 8, 4, 64]
    d.stride_o[:] = 8 * 64, 64, 2 * 8 * 64       # [H, B, L, 64]
    d.stride_dq[:] = 64, 2 * 64, 2 * 8 * 64      # [H, L, B, 64]
    assert lib.ssm_linattn_fwd(d, *[FAKE] * 3, None, *[FAKE] * 4, None, 0, None) == -1 and "log_decay" in err(lib)
    d.stride_o[:] = 8 * 4 * 64, 64, 3 * 64       # the heads of a token over the next tokens
    assert lib.ssm_linattn_fwd(d, *[FAKE] * 8, None, 0, None) == -1 and "overlaps" in err(lib)
    d.stride_o[:] = 7 * 4 * 64, 4 * 64, 64       # a batch row over the end of the one before
    assert lib.ssm_linattn_fwd(d, *[FAKE] * 8, None, 0, None) == -1 and "overlaps" in err(lib)
    r = rope_desc()
    r.stride_k_out[:] = 8 * 2 * 64 - 8, 2 * 64, 64
    assert lib.ssm_rope_fwd(r, *[FAKE] * 6, None) == -1 and "k_out" in err(lib)


def test_states_of_the_gradient_may_not_be_shared(lib):
    d = la_desc(g=4)
    args = dict.fromkeys(["q", "k", "v", "log_decay", "state_in", "lengths", "do", "dstate_out", "dq", "dk", "dv"], FAKE)
    args["state_in"] = FAKE + 256
    assert lib.ssm_linattn_bwd(d, *args.values(), FAKE + 256, None, 0, None) == -1 and "state_in" in err(lib)


def test_outputs_over_inputs_are_refused(lib):
    """By address or, with the same strides, by any value in common.  (What is taken, views of one buffer
    side by side among it, is launched, and so tested with real buffers on a GPU.)"""
    E = 2                                     # bytes a value
    at = lambda i: FAKE + E * i               # noqa: E731
    d = la_desc(g=4)                          # [2, 8, 4, 64] each
    row, n = 4 * 64, 2 * 8 * 4 * 64

    def fwd(d, q, k, v, o, si=FAKE + (1 << 30), so=FAKE + (2 << 30)):
        return lib.ssm_linattn_fwd(d, q, k, v, FAKE, si, None, o, so, None, 0, None)

    far = (at(0), at(2 * n), at(4 * n))
    for i, name in enumerate("qkv"):
        for off in (0, 63, -63, 64, row, -row, n - 1, 1 - n):
            rc = fwd(d, *far, far[i] + E * off)
            assert rc == -1 and "o lies over " + name in err(lib), (name, off)
    w = la_desc(g=4)                          # q, k, v and o side by side in rows of 16 heads
    for f in ("stride_q", "stride_k", "stride_v", "stride_o"):
        getattr(w, f)[:] = 8 * 16 * 64, 16 * 64, 64
    side = [at(4 * 64 * i) for i in range(4)]
    assert fwd(w, *side[:3], side[2] + E * 64) == -1 and "over v" in err(lib)        # three of v's heads
    assert fwd(w, *side[:3], side[3] + E * 64) == -1 and "over q" in err(lib)        # the next token's q
    assert fwd(d, *far, at(6 * n), si=FAKE + (1 << 30), so=FAKE + (1 << 30) + 4) == -1 and "state_out" in err(lib)
    names = ["q", "k", "v", "log_decay", "state_in", "lengths", "do", "dstate_out", "dq", "dk", "dv", "dstate_in"]
    ok = dict(zip(names, [at(2 * n * i) for i in range(12)])) | dict(state_in=FAKE + (1 << 30), lengths=None,
                                                                     dstate_out=FAKE + (2 << 30), dstate_in=FAKE + (3 << 30))

    def bwd(**kw):
        return lib.ssm_linattn_bwd(d, *[(ok | kw)[x] for x in names], None, 0, None)

    for out in ("dq", "dk", "dv"):
        for over in ("q", "k", "v", "do"):
            assert bwd(**{out: ok[over]}) == -1 and f"{out} lies over {over}" in err(lib)
        for other in {"dq", "dk", "dv"} - {out}:
            assert bwd(**{out: ok[other] + E * row}) == -1 and "lies over" in err(lib)
    assert bwd(dstate_in=ok["dstate_out"] + 16) == -1 and "dstate" in err(lib)
    one = la_desc(seqlen=1, g=4)
    assert lib.ssm_linattn_step(one, *far, FAKE, FAKE + (1 << 30), far[2], None) == -1 and "over v" in err(lib)
    x, y8, scales, rstd = (FAKE + (i << 30) for i in range(4))      # 4 rows of 256
    m, far = norm_desc(), FAKE + (5 << 30)

    def norm(d, r, y=far, res=FAKE + (6 << 30)):
        return lib.ssm_rmsnorm_fwd(d, x, res, None, r, y, y8, scales, rstd, None)

    for off in (1, -1, 255, 256, -256, 1023):
        assert norm(m, x + E * off) == -1 and "r lies over x" in err(lib)
        assert norm(m, far, far + E * off) == -1 and "y lies over r" in err(lib)
        assert norm(m, far, x + E * off) == -1 and "y lies over x" in err(lib)
        assert norm(m, far + E * off, far + (1 << 25), far) == -1 and "r lies over residual" in err(lib)
        b = [far, x, FAKE, rstd, far + (1 << 26)]
        for i, name in ((0, "dy"), (1, "r"), (4, "dr")):
            assert lib.ssm_rmsnorm_bwd(m, *b[:2], None, rstd, b[4], b[i] + E * off, None, None, 0, None) == -1
            assert "dx lies over " + name in err(lib)
    assert norm(m, far, far) == -1 and "y lies over r" in err(lib)
    assert norm(norm_desc(stride_r=512), x) == -1 and "r lies over x" in err(lib)     # in place, another stride
    far = (at(0), at(2 * n), at(4 * n))
    r = rope_desc(hq=4, hk=4)

    def rope(d, q, k, qo, ko):
        return lib.ssm_rope_fwd(d, q, k, FAKE, None, qo, ko, None)

    assert rope(r, far[0], far[1], far[1], far[0]) == -1 and "q_out lies over k" in err(lib)
    assert rope(r, far[0], far[1], far[0] + E * row, far[1]) == -1 and "over q" in err(lib)
    assert rope(r, far[0], far[1], far[2], far[2] + E) == -1 and "k_out" in err(lib)
    r.stride_q_out[:] = 8 * 4 * 64, 64, 8 * 64                             # in place, other strides
    assert rope(r, far[0], far[1], far[0], far[1]) == -1 and "over q" in err(lib)


def test_nothing_to_do_is_no_error(lib):
    assert lib.ssm_linattn_fwd(la_desc(seqlen=0), *[None] * 8, None, 0, None) == 0
    assert lib.ssm_rope_fwd(rope_desc(hq=0, hk=0), *[None] * 6, None) == 0


def test_host_tensors_refused():
    torch = pytest.importorskip("torch")
    from selective_diagonal_state_b200 import layer
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        layer.rmsnorm(x)
    q = torch.zeros(1, 3, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        layer.rope(q, q, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        layer.linattn(q, q, q, torch.zeros(2))


def test_row_strides():
    """Of evenly spaced rows, of which there may be none whatever the leading dimensions."""
    torch = pytest.importorskip("torch")
    from selective_diagonal_state_b200 import layer
    for shape, step in (((5, 8), 8), ((2, 3, 8), 8), ((2, 0, 8), 8), ((0, 3, 8), 8), ((2, 3, 0, 8), 8), ((8,), 8), ((1, 1, 8), 8)):
        assert layer._rows(torch.empty(shape), "x", 8) == step
    assert layer._rows(torch.empty(4, 3, 16)[..., :8], "x", 8) == 16
    assert layer._rows(torch.empty(4, 3, 8)[:, 1], "x", 8) == 24
    assert layer._rows(torch.empty(1, 8).expand(6, 8), "x", 8) == 0
    with pytest.raises(ValueError, match="evenly"):
        layer._rows(torch.empty(4, 3, 8)[:, :2], "x", 8)
    for shape in ((2, 3, 8), (2, 0, 8), (0, 3), (1, 1, 8), (2, 1, 4, 1)):      # the helpers' outputs are dense
        out = torch.empty_like(layer._like(shape, torch.float32, "cpu"))
        assert out.shape == shape and out.stride() == torch.empty(shape).stride()


def test_tensors_without_memory_are_refused_and_leave_nothing_behind():
    """A call under a mode that makes fake tensors keeps no plan: a later call of the same layout
    would take its outputs from fake prototypes."""
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode

    from selective_diagonal_state_b200 import layer
    before = dict(layer._PLANS)
    with FakeTensorMode():
        x = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
        q, dec = torch.empty(1, 3, 2, 8, device="cuda"), torch.empty(2, device="cuda")
        freq, state = torch.empty(4, dtype=torch.float64, device="cuda"), torch.empty(1, 2, 8, 8, device="cuda")
        for call in (lambda: layer.rmsnorm(x), lambda: layer.rmsnorm(x[:0], quant="row"),
                     lambda: layer.rmsnorm_backward(x, x, None, x[:, 0].float()), lambda: layer.rope(q, q, freq),
                     lambda: layer.linattn(q, q, q, dec), lambda: layer.linattn_backward(q, q, q, dec, q),
                     lambda: layer.linattn_step(q[:, :1], q[:, :1], q[:, :1], dec, state)):
            with pytest.raises(ValueError, match="memory"):
                call()
    assert layer._PLANS == before


def test_reference_gradients_against_differences():
    """The 64-bit gradients the kernels are held to, against central differences."""
    g = np.random.default_rng(0)
    B, L, H, G, dk, dv = 2, 5, 4, 2, 3, 2
    q, k, v = g.standard_normal((B, L, H, dk)), g.standard_normal((B, L, G, dk)), g.standard_normal((B, L, G, dv))
    s0, ds, do = g.standard_normal((B, H, dk, dv)), g.standard_normal((B, H, dk, dv)), g.standard_normal((B, L, H, dv))
    dec, n, scale = -np.exp(g.uniform(-3, 0.5, H)), np.array([5, 3]), 0.7

    def loss(q, k, v, s0):
        o, S = R.linattn(q, k, v, dec, scale, s0, n)
        return (o * do).sum() + (S * ds).sum()

    args = [q, k, v, s0]
    for i, got in enumerate(R.linattn_bwd(q, k, v, dec, scale, do, s0, ds, n)):
        flat = args[i].reshape(-1)
        for j in g.choice(flat.size, 12, replace=False):
            h, old = 1e-5, flat[j]
            flat[j] = old + h
            up = loss(*args)
            flat[j] = old - h
            down = loss(*args)
            flat[j] = old
            assert got.reshape(-1)[j] == pytest.approx((up - down) / (2 * h), rel=1e-6, abs=1e-8)
    x, w, dy = g.standard_normal((3, 6)), g.standard_normal(6), g.standard_normal((3, 6))
    r, y, rstd = R.norm(x, None, w, 1e-3, None)
    dx, dw = R.norm_bwd(dy, r, w, rstd, None)
    f = lambda x, w: (R.norm(x, None, w, 1e-3, None)[1] * dy).sum()  # noqa: E731
    for a, got in ((x, dx), (w, dw)):
        for j in range(a.size):
            old = a.flat[j]
            a.flat[j] = old + 1e-6
            up = f(x, w)
            a.flat[j] = old - 1e-6
            down = f(x, w)
            a.flat[j] = old
            assert got.flat[j] == pytest.approx((up - down) / 2e-6, rel=1e-6, abs=1e-8)
    xr, fr = g.standard_normal((1, 4, 2, 6)), np.array([1.0, 0.1])
    pos = np.array([[0, 5, -3, 1 << 33]])
    for lay in ("half", "pairs"):
        a, b = R.rope(xr, fr, pos, lay, 1.3), g.standard_normal(xr.shape)
        back = R.rope(b, fr, pos, lay, 1.3, -1.0)
        assert (a * b).sum() == pytest.approx((xr * back).sum())     # the adjoint
