"""The integer form and the orthogonalised update at the ends of what their documentation
allows: arrays past 2^31 elements, the longest sides, the longest list, graphs that share a
workspace, calls at once on two streams, outputs at odd addresses."""
import ctypes
import math

import pytest
import torch

from integer_util import (DEV, F32, HALF, TINY, check_backward, check_orthogonal, check_product, gen, tokens, weak_of,
                          weights)

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _backward_into(L, x, dy, dx, dw, ws):
    """linear_integer_backward with the caller's outputs: the C entry."""
    owq = _owq()
    c, _ = owq._integer_layer(L)
    owq._check(owq.lib().owq_linear_integer_backward(ctypes.byref(c), x.data_ptr(), dy.data_ptr(), x.shape[0], dx.data_ptr(),
                                                     dw.data_ptr(), ws.data_ptr(), ws.numel(),
                                                     torch.cuda.current_stream().cuda_stream), "owq_linear_integer_backward")


def _layer(N, K, k, seed=0):
    g = gen(seed)
    idx = weak_of(g, K, k)
    return _owq().pack_integer(weights(g, N, K), idx), idx


@pytest.mark.parametrize("M,N,K", [(270000, 40, 8192), (270000, 8200, 32)])
def test_product_past_31_bits(M, N, K):
    owq = _owq()
    L, idx = _layer(N, K, 5)
    x = torch.randn(M, K, generator=gen(1), device=DEV, dtype=torch.float16)
    y = owq.linear_integer(L, x)
    rows = torch.tensor([0, 1, 255, 256, 131071, 131072, 262143, 262144, 265000, M - 2, M - 1], device=DEV)
    check_product(L, x[rows], y[rows])


@pytest.mark.parametrize("M,N,K", [(270000, 40, 8192), (270000, 8200, 32)])
def test_backward_past_31_bits(M, N, K):
    owq = _owq()
    L, idx = _layer(N, K, 5)
    g = gen(2)
    x = torch.randn(M, K, generator=g, device=DEV, dtype=torch.float16)
    dy = torch.randn(M, N, generator=g, device=DEV, dtype=torch.float16)
    dx, dw = owq.linear_integer_backward(L, x, dy)
    rows = torch.tensor([0, 127, 128, 131072, 262143, 262144, 265000, M - 1], device=DEV)
    check_backward(L, x[rows], dy[rows], dx[rows], None)
    want = torch.zeros(N, 5, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for m in range(0, M, 30000):
        d, xw = dy[m:m + 30000].double().t().contiguous(), x[m:m + 30000][:, idx.long()].double()
        want += d @ xw
        mag += d.abs() @ xw.abs()
    assert bool(((dw.double() - want).abs() <= M * F32 * mag).all())
    # the sum's roundings are independent of one another: far inside the bound above
    assert float((dw.double() - want).pow(2).mean().sqrt()) <= 16 * F32 * float(mag.pow(2).mean().sqrt())


# the tiled product: whole tiles, halves, one and several parts of K, uneven last parts
@pytest.mark.parametrize("M,N,K,k", [(1025, 1, 32, 0), (1025, 200, 96, 7), (1290, 513, 1056, 9), (1025, 40, 4128, 33),
                                     (1300, 1031, 4096, 32), (257, 2048, 11008, 30), (300, 4096, 11008, 86), (513, 4100, 4096, 5),
                                     (129, 8300, 8224, 63), (65, 16500, 160, 40), (2048, 5000, 416, 12)])
def test_tiled_product(M, N, K, k):
    owq = _owq()
    L, idx = _layer(N, K, k, seed=M)
    x = tokens(gen(M + N), M, K, idx)
    x[M // 2] = 0
    check_product(L, x, owq.linear_integer(L, x))


@pytest.mark.parametrize("N,K,M", [(768, 768, 1024), (4096, 4096, 384), (4096, 4096, 385), (4096, 11008, 128), (16384, 64, 100)])
def test_on_both_sides_of_the_streaming_limit(N, K, M):
    owq = _owq()
    L, idx = _layer(N, K, 6, seed=N + K)
    x = tokens(gen(M), M, K, idx)
    y = owq.linear_integer(L, x)
    check_product(L, x, y)
    # a token's outputs do not depend on the other tokens of the call
    assert torch.equal(owq.linear_integer(L, x.flip(0).contiguous()).flip(0), y)


@pytest.mark.parametrize("r,c", [(1 << 20, 3), (3, 1 << 20), (1 << 20, 100), (100, 1 << 20), (1, 1 << 20)])
def test_longest_sides(r, c):
    owq = _owq()
    G = torch.randn(r, c, generator=gen(r % 97 + c % 89), device=DEV)
    out, = owq.orthogonalize([G], outs=[torch.empty_like(G)])
    check_orthogonal(G, out, 5, QUINTIC, 1e-7, 1.0)


def test_update_past_31_bits():
    owq = _owq()
    r, c = 1 << 20, 2100
    G = torch.empty(r, c, dtype=torch.float16, device=DEV)
    for m in range(0, r, 1 << 17):
        G[m:m + (1 << 17)].normal_(0, 1, generator=gen(m >> 17))
    out, = owq.orthogonalize([G], outs=[torch.empty_like(G)])
    S, sq = torch.zeros(c, c, dtype=torch.float64, device=DEV), 0.0
    for m in range(0, r, 1 << 17):
        d = G[m:m + (1 << 17)].double()
        S += d.t().contiguous() @ d
        sq += float(d.pow(2).sum())
    a, b, q = QUINTIC
    inv = 1.0 / (math.sqrt(sq) + 1e-7)
    eye = torch.eye(c, dtype=torch.float64, device=DEV)
    S, F = S * inv * inv, eye
    for _ in range(5):
        Q = a * eye + b * S + q * S @ S
        F, S = F @ Q, S @ Q @ Q
    rows = torch.tensor([0, 1, 131072, 1022613, 1022614, 1040000, r - 1], device=DEV)
    want = G[rows].double() @ F * inv
    err, size = float((out[rows].double() - want).pow(2).mean().sqrt()), float(want.pow(2).mean().sqrt())
    assert err <= (2.0 ** -24 * a ** 5 + HALF + TINY / size) * size


def test_longest_list():
    owq = _owq()
    g = gen(11)
    shapes = [(1 + i * 7 % 61, 1 + i * 5 % 97) for i in range(4090)] + [(150, 140)] * 6
    Gs = [torch.randn(r, c, generator=g, device=DEV) for r, c in shapes]
    outs = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs])
    for i in list(range(0, 4090, 409)) + [4089, 4090, 4095]:
        alone, = owq.orthogonalize([Gs[i]], outs=[torch.empty_like(Gs[i])])
        assert torch.equal(alone, outs[i]), i
        check_orthogonal(Gs[i], outs[i], 5, QUINTIC, 1e-7, 1.0)


@pytest.mark.parametrize("M", [12, 80, 300])
def test_graphs_that_share_a_workspace(M):
    """Three calls captured into graphs of their own, on one workspace, replayed in turn
    and in any order, with eager work on it in between."""
    owq = _owq()
    N, K, k = 515, 1056, 9
    L, idx = _layer(N, K, k)
    g = gen(M)
    x, dy = tokens(g, M, K, idx), torch.randn(M, N, generator=g, device=DEV).half()
    G = [torch.randn(N, k, generator=g, device=DEV), torch.randn(300, 130, generator=g, device=DEV)]
    need = max(owq.linear_integer_workspace_bytes(N, K, k, M), owq.linear_integer_backward_workspace_bytes(N, K, k, M),
               owq.orthogonalize_workspace_bytes([(N, k), (300, 130)]))
    ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    ws = ws[(-ws.data_ptr()) % 256:][:need]
    y, dx = torch.empty(M, N, dtype=torch.float16, device=DEV), torch.empty_like(x)
    dw, outs = torch.empty(N, k, device=DEV), [torch.empty_like(t) for t in G]
    calls = [lambda: owq.linear_integer(L, x, y=y, workspace=ws),
             lambda: _backward_into(L, x, dy, dx, dw, ws),
             lambda: owq.orthogonalize(G, outs=outs, workspace=ws)]
    graphs = []
    for call in calls:
        call()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for i, order in enumerate([(0, 1, 2), (2, 1, 0), (1, 0, 2), (1, 2, 0)]):
        for t in (y, dx, dw, *outs):
            t.zero_()
        for n in order:
            graphs[n].replay()
            if i % 2:
                ws.fill_(0xff)
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw, *outs)]
        want = [owq.linear_integer(L, x), *owq.linear_integer_backward(L, x, dy),
                *owq.orthogonalize(G, outs=[torch.empty_like(t) for t in G])]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        x.mul_(0.75), dy.mul_(-0.5)
        for t in G:
            t.mul_(1.5)


def test_calls_at_once():
    """Two streams, each with workspaces and outputs of its own, on the same inputs."""
    owq = _owq()
    N, K, k, M = 2000, 2080, 20, 300
    L, idx = _layer(N, K, k)
    g = gen(21)
    x, dy = tokens(g, M, K, idx), torch.randn(M, N, generator=g, device=DEV).half()
    G = [torch.randn(N, k, generator=g, device=DEV) for _ in range(30)] + [torch.randn(400, 300, generator=g, device=DEV)]
    want = [owq.linear_integer(L, x), *owq.linear_integer_backward(L, x, dy),
            *owq.orthogonalize(G, outs=[torch.empty_like(t) for t in G])]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                a = owq.linear_integer(L, x)
                b = owq.linear_integer_backward(L, x, dy)
                c = owq.orthogonalize(G, outs=[torch.empty_like(t) for t in G])
                got[n].append([a, *b, *c])
    torch.cuda.synchronize()
    for per in got:
        for one in per:
            assert all(torch.equal(a, b) for a, b in zip(one, want))


@pytest.mark.parametrize("M", [1, 9, 90, 300])
def test_outputs_at_odd_addresses(M):
    owq = _owq()
    N, K, k = 517, 1056, 9
    L, idx = _layer(N, K, k)
    g = gen(M + 30)
    x, dy = tokens(g, M, K, idx), torch.randn(M, N, generator=g, device=DEV).half()
    want, (wx, ww) = owq.linear_integer(L, x), owq.linear_integer_backward(L, x, dy)
    room = [torch.full((M * w + 40,), 7.0, dtype=t, device=DEV)
            for w, t in ((N, torch.float16), (K, torch.float16), (N, torch.float16))]
    y, dx, d = (r[19:19 + M * w].view(M, w) for r, w in zip(room, (N, K, N)))
    dwr = torch.full((N * k + 8,), 7.0, device=DEV)
    dw = dwr[3:3 + N * k].view(N, k)
    d.copy_(dy)
    owq.linear_integer(L, x, y=y)
    ws = torch.empty(owq.linear_integer_backward_workspace_bytes(N, K, k, M), dtype=torch.uint8, device=DEV)
    _backward_into(L, x, d, dx, dw, ws)
    assert torch.equal(y, want) and torch.equal(dx, wx) and torch.equal(dw, ww)
    for r in room:
        assert bool((r[:19] == 7).all()) and bool((r[-21:] == 7).all())
    assert bool((dwr[:3] == 7).all()) and bool((dwr[-5:] == 7).all())


def test_a_weak_column_of_every_kind_of_place():
    """Weak columns at the first and last place of every tile and step, all columns of one
    tile, and the rest of the row dense."""
    owq = _owq()
    N, K = 300, 2080
    idx = torch.tensor(sorted(set(range(0, 2080, 64)) | set(range(63, 2080, 64)) | set(range(1024, 1056)) | {2079}),
                       dtype=torch.int32, device=DEV)
    g = gen(31)
    L = owq.pack_integer(weights(g, N, K), idx)
    for M in (1, 4, 5, 64, 65, 257):
        x, dy = tokens(g, M, K, idx), torch.randn(M, N, generator=g, device=DEV).half()
        check_product(L, x, owq.linear_integer(L, x))
        check_backward(L, x, dy, *owq.linear_integer_backward(L, x, dy))
