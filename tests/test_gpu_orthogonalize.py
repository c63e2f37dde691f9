"""The orthogonalised update against the definition in 64 bits: both forms (short sides
up to 96 and longer), tall and wide, one row, one column, odd sizes, both types, low rank,
zeros, values that are not finite, many matrices at once, in place, streams and graphs."""
import math

import pytest
import torch

from integer_util import DEV, check_orthogonal, gen, newton_schulz

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _matrix(g, r, c, dt=torch.float32, size=0.01):
    q = min(r, c, 8)
    strong = torch.randn(r, q, generator=g, device=DEV) * (4.0 * 0.6 ** torch.arange(q, device=DEV))
    return (size * (strong @ torch.randn(q, c, generator=g, device=DEV)
                    + torch.randn(r, c, generator=g, device=DEV))).to(dt)


SHAPES = [(1, 1), (1, 7), (7, 1), (5, 5), (16, 16), (17, 33), (4096, 6), (6, 4099), (4097, 32), (33, 500), (64, 64), (65, 70),
          (2000, 86), (86, 1111), (96, 96), (97, 97), (97, 1000), (1000, 130), (221, 2048), (3000, 221), (384, 320)]


@pytest.mark.parametrize("dt", [torch.float32, torch.float16])
@pytest.mark.parametrize("r,c", SHAPES)
def test_update(r, c, dt):
    owq = _owq()
    G = _matrix(gen(r * 31 + c), r, c, dt)
    keep = G.clone()
    scale = 0.3 * math.sqrt(max(1.0, r / c))
    out = torch.empty_like(G)
    assert owq.orthogonalize([G], outs=[out], scales=[scale])[0] is out
    assert torch.equal(G, keep)
    check_orthogonal(G, out, 5, QUINTIC, EPS, scale)


@pytest.mark.parametrize("r,c", [(300, 40), (150, 120)])
@pytest.mark.parametrize("steps", [1, 2, 3, 10])
def test_steps_and_coefficients(r, c, steps):
    owq = _owq()
    G = _matrix(gen(steps), r, c)
    for coef in (QUINTIC, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)):
        out, = owq.orthogonalize([G], outs=[torch.empty_like(G)], steps=steps, coefficients=coef)
        check_orthogonal(G, out, min(steps, 5), coef, EPS, 1.0) if steps <= 5 else None
        if steps == 10 and coef[0] < 2:
            want = newton_schulz(G, steps, coef, EPS, 1.0)
            err = float((out.double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt())
            assert err <= 2.0 ** -24 * coef[0] ** steps


@pytest.mark.parametrize("r,c", [(4096, 32), (64, 3000), (1000, 200)])
def test_singular_values_go_to_one(r, c):
    owq = _owq()
    G = torch.randn(r, c, generator=gen(5), device=DEV)
    O, = owq.orthogonalize([G], outs=[torch.empty_like(G)], steps=16, coefficients=(1.875, -1.25, 0.375))
    s = torch.linalg.svdvals(O.double())
    assert float((s - 1).abs().max()) < 1e-5
    U, _, V = torch.linalg.svd(G.double(), full_matrices=False)
    assert float((O.double() - U @ V).abs().max()) < 1e-5


def test_directions_far_below_the_largest():
    """Singular values down to 1e-4 of the largest keep their precision in the short form."""
    owq = _owq()
    g = gen(9)
    U, _ = torch.linalg.qr(torch.randn(3000, 64, generator=g, device=DEV).double())
    V, _ = torch.linalg.qr(torch.randn(64, 64, generator=g, device=DEV).double())
    G = (U * torch.logspace(0, -4, 64, device=DEV, dtype=torch.float64) @ V.t()).float()
    O, = owq.orthogonalize([G], outs=[torch.empty_like(G)])
    want = newton_schulz(G, 5, QUINTIC, EPS, 1.0)
    err = torch.linalg.matrix_norm(O.double() - want, 2)
    # fp32 products of G with a factor of norm up to a^5: 2^-24 485 of |G|, twice
    assert float(err) <= 2 * 2.0 ** -24 * 485


def test_many_at_once_is_each_alone():
    owq = _owq()
    g = gen(3)
    Gs = [_matrix(g, *SHAPES[i % len(SHAPES)], torch.float16 if i % 3 == 0 else torch.float32) for i in range(150)]
    Gs += [torch.empty(0, 5, device=DEV), torch.empty(40, 0, device=DEV, dtype=torch.float16)]
    scales = [0.5 + 0.01 * i for i in range(len(Gs))]
    outs = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs], scales=scales)
    for i in list(range(0, 150, 7)) + [0, 149]:
        alone, = owq.orthogonalize([Gs[i]], outs=[torch.empty_like(Gs[i])], scales=[scales[i]])
        assert torch.equal(alone, outs[i]), i
        check_orthogonal(Gs[i], outs[i], 5, QUINTIC, EPS, scales[i])


@pytest.mark.parametrize("r,c", [(500, 40), (40, 500), (700, 110), (110, 700)])
@pytest.mark.parametrize("dt", [torch.float32, torch.float16])
def test_in_place_at_odd_addresses(r, c, dt):
    owq = _owq()
    G = _matrix(gen(r + c), r, c, dt)
    want, = owq.orthogonalize([G], outs=[torch.empty_like(G)])
    room = torch.full((r * c + 33,), 5.0, dtype=dt, device=DEV)
    mine = room[17:17 + r * c].view(r, c)
    mine.copy_(G)
    assert owq.orthogonalize([mine])[0] is mine
    assert torch.equal(mine, want)
    assert bool((room[:17] == 5).all()) and bool((room[17 + r * c:] == 5).all())


def test_zeros_and_values_that_are_not_finite():
    owq = _owq()
    g = gen(4)
    for r, c in [(300, 20), (20, 300), (300, 130)]:
        good = _matrix(g, r, c)
        alone, = owq.orthogonalize([good], outs=[torch.empty_like(good)])
        for bad in (float("inf"), float("-inf"), float("nan")):
            G = _matrix(g, r, c)
            G[r // 2, c // 2] = bad
            zero = torch.zeros(r, c, device=DEV)
            outs = owq.orthogonalize([good, G, zero], outs=[torch.empty_like(good) for _ in range(3)])
            assert torch.equal(outs[0], alone)
            assert bool(torch.isnan(outs[1]).all())
            assert bool((outs[2] == 0).all())


def test_large_and_small_values():
    owq = _owq()
    g = gen(6)
    for r, c in [(300, 20), (300, 130)]:
        for size in (1e-18, 1e17):
            G = _matrix(g, r, c, size=size)
            out, = owq.orthogonalize([G], outs=[torch.empty_like(G)], eps=1e-30)
            check_orthogonal(G, out, 5, QUINTIC, 1e-30, 1.0)


def test_stream_graph_and_workspace():
    owq = _owq()
    g = gen(8)
    shapes = [(500, 32), (64, 300), (200, 86), (300, 130)]
    Gs = [_matrix(g, r, c) for r, c in shapes]
    outs = [torch.empty_like(t) for t in Gs]
    need = owq.orthogonalize_workspace_bytes(shapes)
    ws = torch.full((need + 512,), 0x3c, dtype=torch.uint8, device=DEV)
    off = (-ws.data_ptr()) % 256
    mine = ws[off:off + need]
    want = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs], workspace=mine)
    assert bool((ws[:off] == 0x3c).all()) and bool((ws[off + need:] == 0x3c).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        owq.orthogonalize(Gs, outs=outs, workspace=mine)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = owq.orthogonalize(Gs, outs=[torch.empty_like(t) for t in Gs])
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for t in Gs:
            t.mul_(-1.5)
