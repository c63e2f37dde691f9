"""The orthogonalised update over its whole range of steps: gradients of
low rank (fewer tokens than weak columns) and with singular values far apart, 1 to 16 steps,
both forms, against the definition in 64 bits and the error that fp32 products make."""
import pytest
import torch

from integer_util import DEV, gen

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)
TAYLOR = (1.875, -1.25, 0.375)
MIDDLE = (3.0, -3.2, 1.2)
EPS = 1e-7


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _exact(G, steps, coefficients, eps, scale=1.0):
    """The definition on the singular values, whose small ones no product drowns."""
    a, b, c = coefficients
    U, s, V = torch.linalg.svd(G.double().cpu(), full_matrices=False)
    x = s / (s.pow(2).sum().sqrt() + eps)
    x = torch.where(x < 1e-14 * x[0], torch.zeros_like(x), x)
    for _ in range(steps):
        x = x * (a + b * x ** 2 + c * x ** 4)
    return (scale * (U * x) @ V).to(DEV)


def _fp32(G, steps, coefficients, eps):
    a, b, c = coefficients
    t = G.shape[0] > G.shape[1]
    X = (G.t() if t else G).float().contiguous()
    X = X / (X.pow(2).sum().sqrt() + eps)
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if t else X


def _low_rank(g, r, c, q):
    return 0.01 * (torch.randn(r, q, generator=g, device=DEV) @ torch.randn(q, c, generator=g, device=DEV))


def _exactly_low_rank(g, r, c, q):
    u, v = (torch.randint(-3, 4, s, generator=g, device=DEV).float() for s in ((r, q), (q, c)))
    v[:, :q] += 8 * torch.eye(q, device=DEV)     # small integers: the product is exact
    return u @ v


def _spread(g, r, c, least):
    s = min(r, c)
    U, _ = torch.linalg.qr(torch.randn(r, s, generator=g, device=DEV).double().cpu())
    V, _ = torch.linalg.qr(torch.randn(c, s, generator=g, device=DEV).double().cpu())
    return ((U * torch.logspace(0, least, s, dtype=torch.float64)) @ V.t()).float().to(DEV)


CASES = {
    "one token of 32": lambda g: _low_rank(g, 512, 32, 1),
    "16 tokens of 32": lambda g: _low_rank(g, 512, 32, 16),
    "8 tokens of 86": lambda g: _low_rank(g, 700, 86, 8),
    "77 tokens of 86": lambda g: _low_rank(g, 700, 86, 77),
    "wide, 5 of 64": lambda g: _low_rank(g, 64, 900, 5),
    "long form, 7 of 120": lambda g: _low_rank(g, 500, 120, 7),
    "exactly 4 of 32": lambda g: _exactly_low_rank(g, 512, 32, 4),
    "exactly 30 of 90": lambda g: _exactly_low_rank(g, 90, 700, 30),
    "down to 1e-4": lambda g: _spread(g, 512, 64, -4),
    "down to 1e-5": lambda g: _spread(g, 512, 32, -5),
    "down to 1e-6": lambda g: _spread(g, 40, 512, -6),
    "long form, down to 1e-6": lambda g: _spread(g, 512, 130, -6),
    "full rank, padded": lambda g: torch.randn(512, 86, generator=g, device=DEV),
    "full rank, far padded": lambda g: torch.randn(512, 17, generator=g, device=DEV),
    "full rank, wide, padded": lambda g: torch.randn(70, 512, generator=g, device=DEV),
}


@pytest.mark.parametrize("coefficients", [QUINTIC, TAYLOR, MIDDLE], ids=["quintic", "taylor", "middle"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_every_number_of_steps(case, coefficients):
    owq = _owq()
    G = CASES[case](gen(len(case)))
    bad = []
    for steps in range(1, 17):
        want = _exact(G, steps, coefficients, EPS)
        got, = owq.orthogonalize([G], outs=[torch.empty_like(G)], steps=steps, coefficients=coefficients)
        size = float(want.norm())
        err, plain = float((got.double() - want).norm()), float((_fp32(G, steps, coefficients, EPS).double() - want).norm())
        # a few times what fp32 products lose, which grows by |a| a step along the directions
        # that are missing or far below the others, and a few roundings of the result
        if not err <= 3 * plain + 2.0 ** -21 * size:
            bad.append((steps, err / size, plain / size))
        # and what is lost stays bounded as the definition's values are (at most 1.21)
        top = float(torch.linalg.matrix_norm(got.double(), 2))
        if not top <= 3.0:
            bad.append((steps, "largest singular value", top))
    assert not bad, bad
