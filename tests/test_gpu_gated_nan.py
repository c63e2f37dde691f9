"""A NaN in the gate layer of a gated block (a tuning step that diverged) reaches every
output it belongs to, with each activation: the step's gradients are NaN, and clipping
them reports a norm that is not finite. What it does not belong to keeps its bits."""
import numpy as np
import pytest

from parity_util import dev, host
from test_gpu_gated import make

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "gelu_tanh", "relu")
N, K = 150, 160


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def _poisoned(gate, how, row):
    bad = dict(gate)
    name = "w_weak" if how == "weak column" else "scales"
    bad[name] = gate[name].clone()
    bad[name][row] = float("nan")
    return bad


def _split(t, row):
    """(what belongs to the row of the layers, the rest), of an output [M][N] or of a gradient [N][k]."""
    a = host(t).astype(np.float32)
    a = a if a.shape[0] == N and a.shape[1] != N else a.T
    return a[row], np.delete(a, row, axis=0)


@pytest.mark.parametrize("how", ["weak column", "step"])
@pytest.mark.parametrize("M", [1, 2, 3, 7, 16, 40, 130, 300])
def test_forward(owq, M, how):
    gate, up, x = make(owq, N, K, 5, 3, M, M)
    row = 77 if M % 2 else 149
    bad = _poisoned(gate, how, row)
    for act in ACTS:
        print(f"gated with NaN: M={M} {act} {how}", flush=True)
        clean = owq.gated(gate, up, dev(x), act=act, save=True)
        got = owq.gated(bad, up, dev(x), act=act, save=True)
        for name, a, b in zip("hgu", got, clean):
            mine, rest = _split(a, row)
            want, other = _split(b, row)
            assert rest.tobytes() == other.tobytes(), (act, name)
            if name == "u":
                assert mine.tobytes() == want.tobytes(), act
            else:
                assert np.isnan(mine).all(), (act, name)


@pytest.mark.parametrize("M", [1, 5, 40, 130])
def test_backward(owq, M):
    import torch
    gate, up, x = make(owq, N, K, 5, 3, M, M + 1)
    dh = (0.01 * np.random.default_rng(M).standard_normal((M, N))).astype(np.float16)
    row, token = 31, M // 2
    for act in ACTS:
        print(f"gated backward with NaN: M={M} {act}", flush=True)
        _, g, u = owq.gated(gate, up, dev(x), act=act, save=True)
        clean = owq.gated_backward(gate, up, dev(x), g, u, dev(dh), act=act)
        bad = g.clone()
        bad[token, row] = float("nan")
        got = owq.gated_backward(gate, up, dev(x), bad, u, dev(dh), act=act)
        dx, want = host(got[0]), host(clean[0])
        assert np.isnan(dx[token].astype(np.float32)).all(), act
        assert np.delete(dx, token, 0).tobytes() == np.delete(want, token, 0).tobytes(), act
        for a, b in zip(got[1:], clean[1:]):
            mine, rest = _split(a, row)
            assert np.isnan(mine).all(), act
            assert rest.tobytes() == _split(b, row)[1].tobytes(), act
        norm = owq.clip_grad_norm([got[1], got[2]], 1.0)
        assert not bool(torch.isfinite(norm).any()), act


def test_relu_of_zero_and_negative(owq):
    """relu of -0, 0 and below is 0, with slope 0; above, the value and slope 1."""
    gate, up, x = make(owq, N, K, 0, 0, 4, 9)
    g = np.array([-3.0, -0.0, 0.0, 2.0], np.float32)[:, None] * np.ones((4, N), np.float32)
    u = np.full((4, N), 0.5, np.float32)
    dh = np.ones((4, N), np.float16)
    dx = host(owq.gated_backward(gate, up, None, dev(g), dev(u), dev(dh), act="relu", want_dw=False)[0])
    assert not dx[:3].any() and dx[3].any()
