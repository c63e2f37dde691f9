"""The orthogonalised update where numbers leave the middle of fp32's range: zeros at any
eps, gradients of subnormal and of huge numbers, scales from 0 to the type's largest."""
import pytest
import torch

from integer_util import DEV, gen, newton_schulz

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


@pytest.mark.parametrize("eps", [1e-7, 1e-30, 1e-38, 1e-150, 1e-200, 1e-300, 5e-324])
@pytest.mark.parametrize("r,c", [(300, 20), (20, 300), (90, 90), (1, 1), (300, 130)])
def test_zeros_at_any_eps(r, c, eps):
    owq = _owq()
    for steps in (1, 5, 16):
        for dt in (torch.float32, torch.float16):
            G = torch.zeros(r, c, device=DEV, dtype=dt)
            out, = owq.orthogonalize([G], outs=[torch.full_like(G, 3.0)], steps=steps, eps=eps, scales=[1e30])
            assert bool((out == 0).all()), (steps, dt)


@pytest.mark.parametrize("r,c", [(300, 20), (33, 500), (300, 86), (300, 130)])
@pytest.mark.parametrize("size", [2.0 ** -146, 1e-42, 1e-36, 1e-20, 1e20, 3e36])
def test_tiny_and_huge_values(r, c, size):
    owq = _owq()
    g = gen(r + c)
    unit = torch.randint(-9, 10, (r, c), generator=g, device=DEV).double()
    G = (unit * size).float()                        # (subnormal for the smallest: taken as it is)
    out, = owq.orthogonalize([G], outs=[torch.empty_like(G)], eps=1e-300)
    want = newton_schulz(G.double(), 5, QUINTIC, 1e-300, 1.0)
    err, top = float((out.double() - want).norm()), float(want.norm())
    assert err <= 2.0 ** -24 * 485 * top, err / top


@pytest.mark.parametrize("r,c", [(300, 20), (33, 500), (300, 130)])
@pytest.mark.parametrize("scale", [0.0, -2.0, 1e-37, 1e30, 3e38])
def test_scales_of_any_size(r, c, scale):
    owq = _owq()
    G = torch.randn(r, c, generator=gen(r), device=DEV)
    one, = owq.orthogonalize([G], outs=[torch.empty_like(G)])
    out, = owq.orthogonalize([G], outs=[torch.empty_like(G)], scales=[scale])
    scale = float(torch.tensor(scale))
    # the scale is rounded with the factor instead of after it: a few roundings, and 2^-149 as such
    err = (out.double() - scale * one.double()).abs()
    assert bool(torch.isfinite(out).all())
    assert float(err.norm()) <= 2.0 ** -21 * float((scale * one.double()).norm()) + 2.0 ** -149 * (r * c) ** 0.5
