"""The block operators at the ends of their size ranges on the GPU: the largest row
counts that a launch holds, and sizes past it, which are refused and named also where
the binding makes the workspace."""
import numpy as np
import pytest

from parity_util import host
from test_gpu_gated import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def _layer(N, K, k, seed):
    """Any codes are a packed layer; the step keeps the sums near one."""
    import torch
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    d = dict(device="cuda:0", generator=g)
    return {"qcodes": torch.randint(-2 ** 31, 2 ** 31, (N, K // 32, 3), dtype=torch.int32, **d),
            "scales": (torch.rand(N, **d) * 0.05 + 0.01).half(),
            "zeros": torch.randint(0, 8, (N,), dtype=torch.uint8, **d),
            "w_weak": torch.randn((N, k), **d).half(),
            "weak_idx": torch.arange(k, dtype=torch.int32, device="cuda:0") * 5}


def _rows(layer, r):
    return {n: t if n == "weak_idx" else t[r].contiguous() for n, t in layer.items()}


@pytest.mark.parametrize("M", [1, 2])
def test_gated_of_2_26_rows(owq, M):
    """2^26 rows: the last rows' codes start past 2^29 bytes, their outputs past 2^26 elements."""
    import torch
    N, K = 2 ** 26, 32
    gate, up = _layer(N, K, 1, 1), _layer(N, K, 2, 2)
    x = (np.random.default_rng(3).standard_normal((M, K))).astype(np.float16)
    print(f"gated: N={N} M={M}", flush=True)
    h = owq.gated(gate, up, torch.from_numpy(x).to("cuda:0"), act="silu")
    torch.cuda.synchronize()
    for r in (slice(0, 300), slice(N // 2 - 150, N // 2 + 150), slice(N - 300, N)):
        check(h[:, r], None, None, reference(_rows(gate, r), _rows(up, r), x, "silu"), str(r))


def test_sizes_past_a_launch_are_named(owq):
    import torch
    gate = _layer(8, 32, 1, 4)

    def z(*shape, dtype=torch.float16):
        return torch.zeros(shape, dtype=dtype, device="cuda:0")

    M = 2 ** 25
    ads = {"A": z(1, 16, 32), "B": z(1, 8, 16), "alpha": z(1, dtype=torch.float32)}
    with pytest.raises(owq.OwqError, match="SHAPE"):
        owq.linear_adapters(gate, ads, z(M, dtype=torch.int32), z(M, 32))
    M = 2 ** 20 + 1
    g = z(M, 8, dtype=torch.float32)
    with pytest.raises(owq.OwqError, match="SHAPE"):
        owq.gated_backward(gate, gate, z(M, 32), g, g, z(M, 8))
