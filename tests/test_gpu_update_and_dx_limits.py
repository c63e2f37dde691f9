"""The orthogonalised update with many steps and the integer form's dx where their ranges
end: many matrices at once, values that are not finite, the longest sides, graphs that share a
workspace, calls at once, the most rows and tokens."""
import math

import pytest
import torch

from integer_dx_util import faults
from integer_util import DEV, gen, newton_schulz, tokens, weak_of, weights

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _matrix(g, r, c, dt=torch.float32):
    return (0.01 * torch.randn(r, c, generator=g, device=DEV)).to(dt)


@pytest.mark.parametrize("steps", [7, 9, 16])
def test_many_at_once_is_each_alone(steps):
    """Gaussian matrices: every singular value is lifted into [0.7, 1.2] and stays."""
    owq = _owq()
    g = gen(steps)
    shapes = [(1, 1), (1, 9), (40, 3), (17, 33), (500, 32), (33, 500), (700, 64), (65, 400), (4099, 86), (96, 800), (300, 130)] * 3
    Gs = [_matrix(g, r, c, torch.float16 if i % 3 == 0 else torch.float32) for i, (r, c) in enumerate(shapes)]
    scales = [0.5 + 0.1 * i for i in range(len(Gs))]
    outs = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs], scales=scales, steps=steps)
    for i, (G, s, o) in enumerate(zip(Gs, scales, outs)):
        alone = G.clone()
        owq.orthogonalize([alone], scales=[s], steps=steps)       # in place
        assert torch.equal(alone, o), i
        if i >= 11:
            continue
        want = newton_schulz(G, steps, QUINTIC, 1e-7, s)
        # a rounding of fp32 is lifted no further than the values themselves are here (by
        # at most 1 over the smallest singular value's share, 200 for these), the result rounded once
        once = 2.0 ** -24 if G.dtype == torch.float32 else 2.0 ** -11 + 2.0 ** -25 / float(want.pow(2).mean().sqrt())
        err = float((o.double() - want).norm() / want.norm())
        assert err <= 200 * 2.0 ** -24 + once, (i, err)


@pytest.mark.parametrize("r,c", [(300, 20), (50, 300), (300, 96)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_with_many_steps(r, c, bad):
    owq = _owq()
    g = gen(r)
    good, G = _matrix(g, r, c), _matrix(g, r, c)
    alone, = owq.orthogonalize([good], outs=[torch.empty_like(good)], steps=12)
    G[r - 1, c - 1] = bad
    outs = owq.orthogonalize([G, good, torch.zeros_like(G)], outs=[torch.empty_like(G) for _ in range(3)], steps=12)
    assert bool(torch.isnan(outs[0]).all()) and torch.equal(outs[1], alone) and bool((outs[2] == 0).all())


@pytest.mark.parametrize("r,c,q", [(1 << 20, 32, 2), (1 << 20, 90, 5), (33, 1 << 20, 1)])
def test_low_rank_of_the_longest_sides_stays_bounded(r, c, q):
    """What the sums over 2^20 leave along missing directions never turns S negative."""
    owq = _owq()
    g = gen(c)
    G = torch.randn(r, q, generator=g, device=DEV) @ torch.randn(q, c, generator=g, device=DEV)
    for steps in (6, 7, 10, 16):
        O, = owq.orthogonalize([G], outs=[torch.empty_like(G)], steps=steps)
        X = O.double() if r > c else O.double().t().contiguous()
        s = torch.linalg.eigvalsh(torch.matmul(X.t().contiguous(), X).cpu()).clamp(min=0).sqrt()
        assert float(s[-1]) <= 3.0, (steps, float(s[-1]))
        assert float(s[-q]) >= 0.5, (steps, float(s[-q]))


def test_steps_of_both_polynomials_in_graphs_on_one_workspace():
    owq = _owq()
    g = gen(3)
    shapes = [(500, 32), (90, 300), (200, 130)]
    Gs = [_matrix(g, r, c) for r, c in shapes]
    ws = torch.empty(owq.orthogonalize_workspace_bytes(shapes), dtype=torch.uint8, device=DEV)
    graphs = {}
    for steps in (5, 9):
        outs = [torch.empty_like(t) for t in Gs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            owq.orthogonalize(Gs, outs=outs, steps=steps, workspace=ws)
        graphs[steps] = graph, outs
    for _ in range(3):
        for steps in (9, 5, 9):
            graph, outs = graphs[steps]
            graph.replay()
            torch.cuda.synchronize()
            want = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs], steps=steps)
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for t in Gs:
            t.mul_(-1.25)


def test_calls_at_once():
    owq = _owq()
    g = gen(4)
    Gs = [[_matrix(g, 3000, 32), _matrix(g, 80, 2000)] for _ in range(4)]
    want = [owq.orthogonalize(G, outs=[torch.empty_like(t) for t in G], steps=5 + 4 * (i % 2)) for i, G in enumerate(Gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Gs]
    got = [owq.orthogonalize(G, outs=[torch.empty_like(t) for t in G], steps=5 + 4 * (i % 2), stream=s)
           for i, (G, s) in enumerate(zip(Gs, streams))]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def _layer(N, K, k):
    g = gen(N + K)
    idx = weak_of(g, K, k)
    return _owq().pack_integer(weights(g, N, K), idx), idx, g


@pytest.mark.parametrize("N,K,k,M", [(1 << 20, 32, 3, 130), ((1 << 20) - 33, 64, 40, 1), (70, 32, 3, 1 << 20)])
def test_dx_of_the_most_rows_and_tokens(N, K, k, M):
    owq = _owq()
    L, idx, g = _layer(N, K, k)
    dy = (torch.randn(M, N, generator=g, device=DEV) * 0.01).half()
    dx, _ = owq.linear_integer_backward(L, None, dy, want_dw=False)
    rows = torch.tensor(sorted({0, 1, M // 2, M - 2, M - 1} & set(range(M))), device=DEV)
    found = faults(L["codes"], L["scales"], L["w_weak"], idx, dy[rows], dx[rows])
    assert not found, found


def test_dx_repeats_itself_at_odd_addresses_and_on_two_streams():
    owq = _owq()
    N, K, k, M = 2731, 1056, 9, 301
    L, idx, g = _layer(N, K, k)
    room = torch.empty(M * N + 1, dtype=torch.float16, device=DEV)
    dy = room[1:].view(M, N)
    dy.copy_(torch.randn(M, N, generator=g, device=DEV) * 0.01)
    want, _ = owq.linear_integer_backward(L, None, dy, want_dw=False)
    assert not faults(L["codes"], L["scales"], L["w_weak"], idx, dy, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [owq.linear_integer_backward(L, None, dy, want_dw=False, stream=s)[0] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)


@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -24])
def test_dx_of_the_smallest_and_largest_gradients(small):
    """Subnormal gradients, and the largest of the type: a power of two per token holds both."""
    owq = _owq()
    L, idx, g = _layer(515, 128, 4)
    dy = (torch.randint(-3, 4, (40, 515), generator=g, device=DEV).float() * small).half()
    dy[7] = (torch.randn(515, generator=g, device=DEV).clamp(-3, 3) * 20000).half()
    L["scales"] *= 2.0 ** -6
    L["w_weak"] *= 2.0 ** -6
    dx, _ = owq.linear_integer_backward(L, None, dy, want_dw=False)
    found = faults(L["codes"], L["scales"], L["w_weak"], idx, dy, dx)
    assert not found, found
    assert math.isfinite(float(dx[7].abs().max()))
