"""An adapter whose alpha is 0 on the GPU: finite ones leave the shared product as it is,
and one that holds a NaN shows in its own tokens' outputs for every token count (0 NaN is
NaN), and in no other token's."""
import numpy as np
import pytest

import adapter_util as au
from parity_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


@pytest.mark.parametrize("zero", [0.0, -0.0, 1e-45], ids=["0", "-0", "subnormal"])
@pytest.mark.parametrize("rank", [5, 12, 24])
@pytest.mark.parametrize("M", [1, 2, 3, 8, 16, 17, 40, 130, 300])
def test_alpha_zero(owq, M, rank, zero):
    N, K, count = 200, 96, 4
    which = np.array([1, 3, -1, 0, 1, 2] * 50, np.int32)[:M]
    layer, x, A, B, alpha = au.beside(N, K, 3, M, rank, count, which, seed=M + rank)
    L, wd, xd = au.device_layer(layer), dev(which), dev(x)

    def run(A, B, alpha):
        return host(owq.linear_adapters(L, {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}, wd, xd))
    none = host(owq.linear_adapters(L, {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}, dev(np.full(M, -1, np.int32)), xd))
    off = alpha.copy()
    off[1] = zero
    y = run(A, B, off)
    mine = which == 1
    assert np.array_equal(y[mine], none[mine])  # (as values: -0 is 0)
    for name in "AB":
        print(f"alpha 0: M={M} rank={rank} NaN in {name}", flush=True)
        bad = {"A": A.copy(), "B": B.copy()}
        bad[name][1] = np.nan
        z = run(bad["A"], bad["B"], off)
        assert np.isnan(z[mine]).all(), name
        assert z[~mine].tobytes() == y[~mine].tobytes(), name
