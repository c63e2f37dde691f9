"""The adapted linear on the GPU where the adapters decide the output: alone with
products that nearly cancel, and beside a layer, within the tolerance that adapter_util
derives."""
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


@pytest.mark.parametrize("make", [au.cancelling, au.beside], ids=["alone", "beside"])
@pytest.mark.parametrize("case", au.CASES, ids=str)
def test_within_the_tolerance(owq, case, make):
    import torch
    N, K, k, M, rank, count = case
    for name in ("mixed", "one", "runs"):
        which = au.requests(name, M, count, np.random.default_rng(M))
        args = make(*case, which, seed=sum(case))
        layer, x, A, B, alpha = args
        print(f"adapters: {case} {make.__name__} {name}", flush=True)
        ws = torch.full((owq.linear_adapters_workspace_bytes(rank, M),), 0xff, dtype=torch.uint8, device="cuda:0")
        y = host(owq.linear_adapters(au.device_layer(layer), {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}, dev(which),
                                     dev(x), workspace=ws)).astype(np.float64)
        want, tol, _ = au.reference(*args, which, make is au.cancelling)
        err = np.abs(y - want)
        assert (err <= tol).all(), f"{name}: exceeds by {np.max(err - tol)}"
        if make is au.cancelling:
            assert not y[which < 0].any()


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("decode", ["vector", "matrix"])
def test_every_decode_kernel(owq, decode, M, monkeypatch):
    monkeypatch.setenv("OWQ_DECODE", decode)
    for products in ("dot2", "mfma"):
        monkeypatch.setenv("OWQ_GEMV_PRODUCTS", products)
        for case in ((131, 64, 2, M, 72, 3), (131, 96, 0, M, 9, 2)):
            which = np.array([1, -1, 0, 1][:M], np.int32)
            for make in (au.cancelling, au.beside):
                args = make(*case, which, seed=M)
                layer, x, A, B, alpha = args
                y = host(owq.linear_adapters(au.device_layer(layer), {"A": dev(A), "B": dev(B), "alpha": dev(alpha)},
                                             dev(which), dev(x))).astype(np.float64)
                want, tol, _ = au.reference(*args, which, make is au.cancelling)
                assert (np.abs(y - want) <= tol).all(), (products, case, make.__name__)
