"""Backward of the integer form's linear against the formula in 64 bits and against
differences of the forward product."""
import pytest
import torch

from integer_util import DEV, check_backward, dequantised, gen, tokens, weak_of, weights

pytestmark = pytest.mark.gpu


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _case(N, K, k, M, seed=0):
    owq = _owq()
    g = gen(seed + N + 3 * K + 5 * k + 7 * M)
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    dy = (torch.randn(M, N, generator=g, device=DEV) * 0.01).half()
    return L, x, dy


@pytest.mark.parametrize("M", [1, 2, 31, 128, 129, 300])
@pytest.mark.parametrize("N,K,k", [(1, 32, 0), (1, 32, 32), (64, 96, 1), (513, 1056, 9), (768, 768, 6), (2731, 160, 40),
                                   (130, 4128, 33)])
def test_gradients(N, K, k, M):
    owq = _owq()
    L, x, dy = _case(N, K, k, M)
    if M > 2:
        dy[1] = 0
    dx, dw = owq.linear_integer_backward(L, x, dy)
    check_backward(L, x, dy, dx, dw)


def test_a_long_layer_and_wide_ranges():
    owq = _owq()
    L, x, dy = _case(11008, 512, 32, 257)
    L["scales"] *= 2.0 ** torch.randint(-6, 7, (11008,), device=DEV).float()  # rows of very different size
    dy *= 2.0 ** torch.randint(-8, 9, (257, 1), device=DEV).half()
    dx, dw = owq.linear_integer_backward(L, x, dy)
    check_backward(L, x, dy, dx, dw)


@pytest.mark.parametrize("M", [5, 200])
def test_parts_alone_and_repeats(M):
    owq = _owq()
    L, x, dy = _case(515, 1056, 9, M)
    dx, dw = owq.linear_integer_backward(L, x, dy)
    only_dx, none = owq.linear_integer_backward(L, None, dy, want_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = owq.linear_integer_backward(L, x, dy, want_dx=False)
    assert none is None and torch.equal(only_dw, dw)
    again = owq.linear_integer_backward(L, x, dy)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_differences():
    """y is linear in the weak weights and, as the backward has it, in x: x times the
    dequantised layer."""
    owq = _owq()
    L, x, dy = _case(96, 128, 5, 6)
    dx, dw = owq.linear_integer_backward(L, x, dy)
    W, xd, d = dequantised(L), x.double(), dy.double()
    loss = lambda v, w: float((d * (v @ w.t())).sum())
    idx = L["weak_idx"].long()
    for i, c in [(0, 0), (50, 3), (95, 4)]:
        E = torch.zeros_like(W)
        E[i, idx[c]] = 1e-3
        diff = (loss(xd, W + E) - loss(xd, W - E)) / 2e-3
        assert abs(diff - float(dw[i, c])) <= 1e-5 * max(1.0, abs(diff))
    for m, j in [(0, 0), (3, 77), (5, int(idx[2]))]:
        E = torch.zeros_like(xd)
        E[m, j] = 1e-3
        diff = (loss(xd + E, W) - loss(xd - E, W)) / 2e-3
        mag = float((d[m].abs() * W[:, j].abs()).sum())
        assert abs(diff - float(dx[m, j])) <= 2.0 ** -10 * (mag + abs(diff))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_gradient_that_is_not_finite_stays_in_its_token(bad):
    owq = _owq()
    L, x, dy = _case(200, 96, 4, 70)
    good, good_w = owq.linear_integer_backward(L, x, dy)
    dy[69, 11] = bad
    dx, dw = owq.linear_integer_backward(L, x, dy)
    assert torch.equal(dx[:69], good[:69]) and not bool(torch.isfinite(dx[69][L["codes"][11] != 0]).any())
    assert torch.equal(dw[:11], good_w[:11]) and torch.equal(dw[12:], good_w[12:])


def test_graph_and_guards():
    owq = _owq()
    N, K, k, M = 515, 1056, 9, 77
    L, x, dy = _case(N, K, k, M)
    need = owq.linear_integer_backward_workspace_bytes(N, K, k, M)
    ws = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device=DEV)
    off = (-ws.data_ptr()) % 256
    mine = ws[off:off + need]
    want = owq.linear_integer_backward(L, x, dy, workspace=mine)
    assert bool((ws[:off] == 0x5a).all()) and bool((ws[off + need:] == 0x5a).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = owq.linear_integer_backward(L, x, dy, workspace=mine)
    for _ in range(3):
        dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        x.mul_(0.5)
        dy.mul_(0.5)
        want = owq.linear_integer_backward(L, x, dy)
