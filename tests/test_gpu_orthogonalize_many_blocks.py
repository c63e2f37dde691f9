"""More matrices than one launch of the orthogonalised update holds blocks."""
import pytest
import torch

from integer_util import DEV, gen

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def test_more_blocks_than_one_launch_holds():
    """4096 columns of 2^20: 2^24 blocks of the last product."""
    owq = _owq()
    count, n = 4096, 1 << 20
    flat = torch.empty(count, n, dtype=torch.float16, device=DEV)
    for i in range(0, count, 64):
        flat[i:i + 64] = torch.randn(64, n, generator=gen(i), device=DEV).half()
    few = [0, 1, 63, 64, 2047, 4094, 4095]
    before = [flat[i].double() for i in few]
    owq.orthogonalize([flat[i].view(n, 1) for i in range(count)], steps=2)
    a, b, c = QUINTIC
    for i, v in zip(few, before):
        x = v.norm() / (v.norm() + EPS)
        f = 1.0
        for _ in range(2):
            p = a + b * x ** 2 + c * x ** 4
            f, x = f * p, x * p
        want = v * f / (v.norm() + EPS)
        # (values of 1e-3: half a step of an fp16 subnormal is 2^-25)
        assert float((flat[i].double() - want).abs().max()) <= 2.0 ** -25 + 2.0 ** -11 * float(want.abs().max())
    # every other column was written too: entries of size 1 / sqrt(n) times the polynomial, none of size 1
    for i in range(0, count, 64):
        assert float(flat[i:i + 64].abs().amax()) < 0.05
