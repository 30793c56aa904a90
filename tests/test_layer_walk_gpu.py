"""Which kernel a linear attention call takes, and the walk's paths that depend on where the
sequences of a padded batch end.  Values against the 64-bit forms with the bounds of
test_layer_gpu.py."""
import numpy as np
import pytest

from selective_diagonal_state_b200 import abi
from tests import layer_ref as R
from tests.test_layer_gpu import DT, close, la_case, la_check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from selective_diagonal_state_b200 import build
    build.build()
    abi.load_library()


@pytest.fixture(scope="module")
def layer():
    from selective_diagonal_state_b200 import layer
    return layer


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    """A bounded wait that gives up is reported behind the call only."""
    yield
    abi.ssm_scan_poll_device_error()


def kernels(call):
    """{kernel: launches} of the calls that `call` makes."""
    abi.ssm_scan_profile_start(64)
    try:
        call()
    finally:
        got = abi.ssm_scan_profile_stop()
    return {name: n for name, (n, _) in got.items()}


def ragged_case(seed, lengths, L, H, G, dk, dv):
    """la_case with these lengths, NaN behind them."""
    T, N = la_case(seed, "bf16", len(lengths), L, H, G, dk, dv, False)
    N["lengths"] = np.array(lengths)
    T["lengths"] = torch.from_numpy(N["lengths"].astype(np.int32)).cuda()
    for name in ("q", "k", "v", "do"):
        for b, n in enumerate(lengths):
            T[name][b, n:] = float("nan")
    return T, N


# the chunk that a sequence ends in is the walk's first (reverse) or its last (forward): the third
# and later ones, whose tiles lie where those of earlier chunks were, at both places
ENDS = [(257, 390, 513, 639, 640, 700), (383, 384, 385, 511, 0, 899), (255, 256, 129, 1, 768, 300)]


@pytest.mark.parametrize("lengths", ENDS)
@pytest.mark.parametrize("H,G,dk,dv", [(2, 1, 128, 64), (3, 3, 16, 24), (2, 2, 64, 128)])
def test_sequences_that_end_in_any_chunk(layer, lengths, H, G, dk, dv):
    L = max(lengths) + (1 if 700 in lengths else 70)
    T, N = ragged_case(L + dk, lengths, L, H, G, dk, dv)
    la_check(layer, T, N, "bf16", dk ** -0.5, True)
    args = [T[x] for x in ("q", "k", "v", "log_decay")]
    # one walk for each head, not cut into segments
    assert kernels(lambda: layer.linattn(*args, lengths=T["lengths"])) == {"k_la_walk": 1}
    back = kernels(lambda: layer.linattn_backward(*args, T["do"], lengths=T["lengths"]))
    assert back == {"k_la_walk": 1} | ({"k_la_group_sum16": 2} if H > G else {})


def test_padded_batch_with_more_walks_than_fit_at_once(layer):
    """24 heads of 4 rows, the lengths in every chunk of the walk, repeated: always the same bits."""
    T, N = ragged_case(5, (257, 390, 513, 639), 700, 24, 24, 16, 24)
    la_check(layer, T, N, "bf16", 0.25, True)
    args = [T[x] for x in ("q", "k", "v", "log_decay")]
    first = layer.linattn(*args, state=T["state"], lengths=T["lengths"], out=torch.zeros(4, 700, 24, 24, dtype=DT["bf16"], device="cuda"))
    for _ in range(20):
        again = layer.linattn(*args, state=T["state"], lengths=T["lengths"], out=torch.zeros_like(first[0]))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("L,dk,dv", [(33, 64, 64), (17, 128, 128), (17, 64, 128), (257, 8, 8)])
def test_shortest_sequences_of_the_walk(layer, L, dk, dv):
    """More than 2048 / head dim tokens take the walk, one less the recurrence."""
    for n, name, tensor in ((L, "k_la_walk", True), (L - 1, "k_la_recurrent", False)):
        T, N = la_case(n, "bf16", 2, n, 2, 1, dk, dv, False)
        la_check(layer, T, N, "bf16", dk ** -0.5, tensor)
        args = [T[x] for x in ("q", "k", "v", "log_decay")]
        assert kernels(lambda: layer.linattn(*args)) == {name: 1}
        assert name in kernels(lambda: layer.linattn_backward(*args, T["do"]))


@pytest.mark.parametrize("L,lengths", [(300, None), (400, (129, 390)), (2600, (1279, 2600))])
def test_values_wider_than_the_keys_may_be(layer, L, lengths):
    """dim_v above 128, three and four slices: the output and the state on tensor cores, the gradient by
    the recurrence (a walk of it would have dim_v state rows)."""
    for dv in (136, 200, 256):
        T, N = ragged_case(dv, lengths, L, 2, 1, 64, dv) if lengths else la_case(dv, "bf16", 2, L, 2, 1, 64, dv, False)
        n = N["lengths"]
        live = np.ones((2, L), bool) if n is None else np.arange(L)[None] < n[:, None]
        out = torch.zeros(2, L, 2, dv, dtype=DT["bf16"], device="cuda")
        o, S = layer.linattn(T["q"], T["k"], T["v"], T["log_decay"], state=T["state"], lengths=T["lengths"], out=out)
        A = {x: np.abs(N[x]) for x in ("q", "k", "v", "state")}
        ro, rS = R.linattn(N["q"], N["k"], N["v"], N["log_decay"], 0.125, N["state"], n)
        ob, sb = R.linattn(A["q"], A["k"], A["v"], N["log_decay"], 0.125, A["state"], n)
        c = (60 * -(-L // 128) + 2 * dv + 16) * R.U32        # as in la_check
        close("o", o, ro, (R.HALF["bf16"] * np.abs(ro) + (R.HALF["bf16"] + c) * ob) * live[..., None, None])
        close("state", S, rS, c * sb)
        args = [T[x] for x in ("q", "k", "v", "log_decay")]
        assert "k_la_walk" in kernels(lambda: layer.linattn(*args, lengths=T["lengths"]))
        assert "k_la_recurrent" in kernels(lambda: layer.linattn_backward(*args, T["do"], lengths=T["lengths"]))


def test_which_calls_are_cut_and_which_take_the_recurrence(layer):
    T, _ = la_case(1, "bf16", 1, 2300, 3, 1, 128, 128, False)
    args = [T[x] for x in ("q", "k", "v", "log_decay")]
    cut = {"k_la_walk_state": 1, "k_la_segments": 1, "k_la_walk": 1}
    assert kernels(lambda: layer.linattn(*args)) == cut
    assert kernels(lambda: layer.linattn(*args, route=abi.LINATTN_RECURRENT)) == {"k_la_recurrent": 1}
    for t, dim, off in (("fp32", 64, 0), ("bf16", 20, 0), ("bf16", 136, 0), ("bf16", 64, 1)):
        x = torch.zeros(1, 300, 2, dim + off, dtype=DT[t], device="cuda")[..., off:]
        assert kernels(lambda: layer.linattn(x, x, x, args[3][:2])) == {"k_la_recurrent": 1}


@pytest.mark.parametrize("B,L,H,G,dk,dv,ragged", [(2, 700, 2, 1, 64, 64, False), (3, 700, 2, 1, 128, 64, True),
                                                  (1, 2300, 3, 1, 128, 128, False), (2, 40, 2, 2, 64, 64, False)])
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_right(layer, B, L, H, G, dk, dv, ragged):
    """With no polls allowed every wait of a walk's warps for one another gives up where it does not pass at
    once; the call ends (its copies and products in flight are still waited for), and the poll reports it."""
    T, _ = la_case(L, "bf16", B, L, H, G, dk, dv, ragged)
    args = [T[x] for x in ("q", "k", "v", "log_decay")]
    calls = (lambda: layer.linattn(*args, state=T["state"], lengths=T["lengths"], out=torch.zeros(B, L, H, dv, dtype=DT["bf16"], device="cuda")),
             lambda: layer.linattn_backward(*args, T["do"], state=T["state"], dstate=T["dstate"], lengths=T["lengths"],
                                            out=[torch.zeros_like(T[x]) for x in ("q", "k", "v")]))
    want = [call() for call in calls]
    abi.ssm_scan_poll_device_error()
    for call, ref in zip(calls, want):
        old = abi.ssm_scan_set_wait_limit(0)
        try:
            call()
            with pytest.raises(abi.SsmError) as e:
                abi.ssm_scan_poll_device_error()
            assert e.value.code == -5        # SSM_ERR_TIMEOUT
        finally:
            abi.ssm_scan_set_wait_limit(old)
        got = call()
        abi.ssm_scan_poll_device_error()     # cleared by the poll above, and nothing new
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
