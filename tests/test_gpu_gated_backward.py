"""Backward of the gated feed-forward block (owq_gated_backward) on the GPU.

Against 64 bits, from the kernel's own inputs (the fp32 g and u it is given):
  da = dh u act'(g) is computed in fp32: the activation's value and slope to
  2^-17 of a, with a = |act'| resp. |act| plus the size of its parts (1 + |g|
  times the logistic or normal factor: taken as 1.2 + |g| where |g| < 20, the
  slope's terms cancel at most to that), so dda = 2^-16 |dh| |u| (1.2 + 0.25 |g|)
  and ddb = 2^-16 |dh| (|act| + 2^-10 |g|), both an upper bound.
  dw: fp32 sums over M tokens of (da + dda) x, at most M + 8 roundings:
    |dw - ref| <= sum_m |x| dda + (M + 8) 2^-24 sum_m |x| (|da| + dda)
  dx: s da is rounded to fp16 relative to its own size (2^-11) or 2^-25 of the
  token's scaled range (2^-25 2^-14 = 2^-39 of the largest |s da|, per row and |q -
  z| <= 7), the sums over 2 N rows and the weak columns are fp32:
    |dx - ref| <= sum |W| dd + (2^-11 + (N + 64) 2^-23) sum |W| (|d| + dd)
                  + 7 * 2 N 2^-39 max |s d| + 2^-11 |ref| + 2^-25
and, end to end with the forward, against differences of the loss in 64 bits."""
import numpy as np
import pytest

import gated_util as gu
from parity_util import dev, host
from test_gpu_gated import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def reference(gate, up, x, g, u, dh, act):
    g, u, dh, x = (t.astype(np.float64) for t in (g, u, dh, x))
    M, N = g.shape
    a, s = gu.act(act, g)
    da, db = dh * u * s, dh * a
    dda = 2.0 ** -16 * np.abs(dh * u) * (1.2 + 0.25 * np.minimum(np.abs(g), 20.0))
    ddb = 2.0 ** -16 * np.abs(dh) * (np.abs(a) + 2.0 ** -10 * np.abs(g))
    out = {}
    dx, tol = 0.0, 0.0
    top = np.zeros((M, 1))
    for name, layer, d, dd in (("dw_gate", gate, da, dda), ("dw_up", up, db, ddb)):
        W = gu.weights(layer)
        xw = x[:, layer["weak_idx"].cpu().numpy()]
        out[name] = (d.T @ xw, dd.T @ np.abs(xw) + (M + 8) * 2.0 ** -24 * ((np.abs(d) + dd).T @ np.abs(xw)))
        dx = dx + d @ W
        tol = tol + dd @ np.abs(W) + (2.0 ** -11 + (N + 64) * 2.0 ** -23) * ((np.abs(d) + dd) @ np.abs(W))
        sc = layer["scales"].cpu().numpy().astype(np.float64)
        top = np.maximum(top, np.max(np.abs(d) * sc, axis=1, keepdims=True))
    tol = tol + 14 * N * 2.0 ** -39 * top + 2.0 ** -11 * np.abs(dx) + 2.0 ** -25
    out["dx"] = (dx, tol)
    return out


def check(got, ref, what):
    for name, t in got.items():
        want, tol = ref[name]
        err = np.abs(host(t).astype(np.float64) - want)
        assert (err <= tol + 1e-30).all(), f"{what} {name}: exceeds by {np.max(err - tol)} (largest {np.abs(want).max()})"


CASES = [
    # N, K, k gate, k up, M
    (1, 32, 0, 1, 1),
    (5, 32, 32, 0, 2),
    (33, 96, 3, 5, 1),
    (130, 4128, 7, 0, 1),
    (700, 544, 40, 33, 3),
    (64, 96, 96, 1, 5),
    (129, 1056, 9, 4, 16),
    (513, 256, 6, 70, 31),
    (1000, 160, 5, 5, 32),
    (127, 96, 2, 0, 33),
    (257, 512, 0, 7, 64),
    (191, 320, 130, 3, 65),
    (300, 992, 9, 9, 129),
    (2050, 288, 0, 0, 200),
    (63, 512, 20, 1, 700),
    (2, 64, 3, 3, 2100),
]


@pytest.mark.parametrize("case", CASES)
def test_against_64_bits(owq, case):
    import torch
    N, K, kg, ku, M = case
    gate, up, x = make(owq, *case, seed=sum(case) + 1)
    rng = np.random.default_rng(5)
    dh = (0.01 * rng.standard_normal((M, N))).astype(np.float16)
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        print(f"gated backward: N={N} K={K} k={kg},{ku} M={M} {act}", flush=True)
        _, g, u = owq.gated(gate, up, dev(x), act=act, save=True)
        ref = reference(gate, up, x, host(g), host(u), dh, act)
        # a workspace of NaN patterns
        ws = torch.full((owq.gated_backward_workspace_bytes(N, K, kg, ku, M),), 0xff, dtype=torch.uint8,
                        device="cuda:0")
        dx, dwg, dwu = owq.gated_backward(gate, up, dev(x), g, u, dev(dh), act=act, workspace=ws)
        torch.cuda.synchronize()
        check({"dx": dx, "dw_gate": dwg, "dw_up": dwu}, ref, act)
        # each output alone: the same bits
        only = owq.gated_backward(gate, up, None, g, u, dev(dh), act=act, want_dw=False)
        assert only[1] is None and only[2] is None and host(only[0]).tobytes() == host(dx).tobytes()
        only = owq.gated_backward(gate, up, dev(x), g, u, dev(dh), act=act, want_dx=False)
        assert only[0] is None
        assert host(only[1]).tobytes() == host(dwg).tobytes() and host(only[2]).tobytes() == host(dwu).tobytes()


@pytest.mark.parametrize("scale", [2.0 ** -20, 1.0, 2.0 ** 12])
def test_gradients_of_any_size(owq, scale):
    """Upstream gradients near fp16's smallest and largest values: dx keeps its relative accuracy."""
    for M in (1, 20, 100):
        gate, up, x = make(owq, 400, 256, 5, 4, M, 11)
        rng = np.random.default_rng(2)
        dh = (rng.standard_normal((M, 400)) * scale).astype(np.float16)
        dh[0] = 0
        if M > 2:
            dh[2] = (dh[2].astype(np.float32) * 2.0 ** -6).astype(np.float16)
        _, g, u = owq.gated(gate, up, dev(x), save=True)
        ref = reference(gate, up, x, host(g), host(u), dh, "silu")
        dx, dwg, dwu = owq.gated_backward(gate, up, dev(x), g, u, dev(dh))
        ok = np.abs(ref["dx"][0]) < 60000
        err = np.abs(host(dx).astype(np.float64) - ref["dx"][0])
        assert (err[ok] <= ref["dx"][1][ok]).all()
        assert not np.isnan(host(dx).astype(np.float32)).any()
        assert not host(dx)[0].any()
        check({"dw_gate": dwg, "dw_up": dwu}, ref, f"scale {scale}")


def test_a_token_keeps_to_itself(owq):
    """Infinities and NaN in one token's gradient change no other token's dx."""
    for M in (3, 40, 130):
        gate, up, x = make(owq, 200, 160, 5, 4, M, 12)
        dh = (0.1 * np.random.default_rng(3).standard_normal((M, 200))).astype(np.float16)
        _, g, u = owq.gated(gate, up, dev(x), save=True)
        a = host(owq.gated_backward(gate, up, dev(x), g, u, dev(dh))[0])
        for bad in (np.inf, np.nan):
            d2 = dh.copy()
            d2[1, 7] = bad
            b = host(owq.gated_backward(gate, up, dev(x), g, u, dev(d2))[0])
            keep = np.arange(M) != 1
            assert a[keep].tobytes() == b[keep].tobytes()
            assert not np.isfinite(b[1].astype(np.float32)).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_against_differences(owq, act):
    """d loss / d x and d loss / d w_weak against central differences of the loss in
    64 bits, loss = sum(h * dh) from the unpacked weights: the differences' own error
    is eps^2 times the third derivative (of order the loss's terms), so 1e-5 of the
    gradient's scale on top of the fp16 and fp32 tolerances (dx: 2e-3, dw: 1e-4)."""
    N, K, M = 48, 64, 4
    gate, up, x = make(owq, N, K, 3, 4, M, 21)
    dh = np.random.default_rng(6).standard_normal((M, N)).astype(np.float16)
    x = (x.astype(np.float32) / 8).astype(np.float16)
    _, g, u = owq.gated(gate, up, dev(x), act=act, save=True)
    dx, dwg, dwu = owq.gated_backward(gate, up, dev(x), g, u, dev(dh), act=act)
    Wg, Wu, x64, d64 = gu.weights(gate), gu.weights(up), x.astype(np.float64), dh.astype(np.float64)

    def loss(Wg, Wu, x):
        return float(np.sum(gu.act(act, x @ Wg.T)[0] * (x @ Wu.T) * d64))

    def diff(make_args, eps=1e-4):
        return (loss(*make_args(eps)) - loss(*make_args(-eps))) / (2 * eps)

    def bumped(a, i, j, e):
        b = a.copy()
        b[i, j] += e
        return b

    scale = np.abs(host(dx).astype(np.float64)).max()
    rng = np.random.default_rng(7)
    for m, j in zip(rng.integers(0, M, 40), rng.integers(0, K, 40)):
        want = diff(lambda e: (Wg, Wu, bumped(x64, m, j, e)))
        assert abs(float(host(dx)[m, j]) - want) <= 2e-3 * scale, (m, j)
    for name, dw, layer in (("gate", dwg, gate), ("up", dwu, up)):
        idx = layer["weak_idx"].cpu().numpy()
        dw = host(dw)
        for i, c in zip(rng.integers(0, N, 40), rng.integers(0, len(idx), 40)):
            want = diff(lambda e: (bumped(Wg, i, idx[c], e), Wu, x64) if name == "gate"
                        else (Wg, bumped(Wu, i, idx[c], e), x64))
            assert abs(float(dw[i, c]) - want) <= 1e-4 * np.abs(dw).max(), (name, i, c)


def test_graph_and_other_stream(owq):
    import torch
    for M in (1, 40, 150):
        gate, up, x = make(owq, 300, 256, 6, 5, M, M + 1)
        dh = dev((0.1 * np.random.default_rng(3).standard_normal((M, 300))).astype(np.float16))
        xd = dev(x)

        def step(stream=None):
            h, g, u = owq.gated(gate, up, xd, save=True, stream=stream)
            return (h,) + owq.gated_backward(gate, up, xd, g, u, dh, stream=stream)

        eager = [host(t).copy() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for rep in range(3):
            for t in outs:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, t in zip(eager, outs):
                assert host(t).tobytes() == a.tobytes()
            for a, t in zip(eager, step()):
                assert host(t).tobytes() == a.tobytes()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = step(side)
        side.synchronize()
        for a, t in zip(eager, other):
            assert host(t).tobytes() == a.tobytes()


def test_training_step(owq):
    """Forward, backward, the global norm and clipping of both weak gradients, the update of
    the weak columns, and a forward with them: against 64 bits."""
    import torch
    M, N, K = 50, 260, 288
    gate, up, x = make(owq, N, K, 8, 5, M, 33)
    dh = (0.1 * np.random.default_rng(3).standard_normal((M, N))).astype(np.float16)
    h, g, u = owq.gated(gate, up, dev(x), save=True)
    ref = reference(gate, up, x, host(g), host(u), dh, "silu")
    dx, dwg, dwu = owq.gated_backward(gate, up, dev(x), g, u, dev(dh))
    grads = [host(dwg).astype(np.float64), host(dwu).astype(np.float64)]
    want = np.sqrt(sum((t ** 2).sum() for t in grads))
    norm = owq.clip_grad_norm([dwg, dwu], 0.5 * want)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    for layer, dw, t in ((gate, dwg, grads[0]), (up, dwu, grads[1])):
        assert (np.abs(host(dw) - 0.5 * t) <= np.abs(t) * 2.0 ** -24 + 1e-30).all()
        layer["w_weak"].sub_(0.01 * dw.half())
    torch.cuda.synchronize()
    from test_gpu_gated import check as check_forward, reference as forward
    h2 = owq.gated(gate, up, dev(x))
    check_forward(h2, None, None, forward(gate, up, x, "silu"), "after the update")
    check({"dx": dx}, ref, "step")
    assert host(h2).tobytes() != host(h).tobytes()
