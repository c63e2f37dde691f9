"""The integer form's sums of codes are exact: sums that cancel give 0 in every form of the
product, and without weak columns an output is off by the three fp32 roundings of the formula
and its own."""
import pytest
import torch

from integer_util import DEV, HALF, TINY, gen, rows_quantised, tokens, weak_of, weights

pytestmark = pytest.mark.gpu
TOKENS = [1, 2, 3, 4, 5, 16, 40, 77, 300]


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("N,K", [(37, 1056), (130, 4096), (50, 11008)])
def test_sums_that_cancel(N, K, M):
    owq = _owq()
    g = gen(N + K + M)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    place = torch.randperm(K, generator=g, device=DEV)
    half = torch.randint(-127, 128, (N, K // 2), generator=g, device=DEV)
    n = torch.randint(-126, 127, (M, K // 2), generator=g, device=DEV)
    n[:, 0] = 127
    codes = torch.empty(N, K, dtype=torch.int8, device=DEV)
    codes[:, place] = torch.cat([half, half], 1).to(torch.int8)
    x = torch.empty(M, K, dtype=torch.float16, device=DEV)
    x[:, place] = (1.25 * torch.cat([n, -n], 1)).half()      # exact: a token's codes are n
    L = {"codes": codes, "scales": 0.001 + 0.01 * torch.rand(N, generator=g, device=DEV),
         "w_weak": torch.zeros(N, 0, dtype=torch.float16, device=DEV), "weak_idx": none}
    assert torch.equal(rows_quantised(x, none)[0], torch.cat([n, -n], 1).double()[:, torch.argsort(place)])
    assert bool((owq.linear_integer(L, x) == 0).all())
    if M <= 16:
        ys = owq.linear_integer_batched([L, L], [x, x])
        assert all(bool((y == 0).all()) for y in ys)


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("N,K", [(37, 1056), (515, 4096), (50, 11008)])
def test_four_roundings(N, K, M):
    owq = _owq()
    g = gen(N + K + M)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    L = owq.pack_integer(weights(g, N, K), none)
    x = tokens(g, M, K, none)
    q, s = rows_quantised(x, none)
    want = (q @ L["codes"].double().t()) * torch.outer(s, L["scales"].double())
    # the sum to fp32, the product of the scales, the product with it: half a step each
    tol = HALF * (1 + HALF) * want.abs() + TINY + 3.01 * 2.0 ** -24 * want.abs()
    err = (owq.linear_integer(L, x).double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
