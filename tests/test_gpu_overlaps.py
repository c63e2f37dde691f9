"""Arrays of the block operators' calls that lie over one another, on the GPU: dx in the
place of an array that has been read, and outputs over inputs, which the binding's calls
refuse too."""
import ctypes

import numpy as np
import pytest

from parity_util import dev, host
from test_gpu_gated import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


@pytest.mark.parametrize("M", [1, 33, 130, 400])
def test_dx_in_the_place_of_an_input(owq, M):
    import torch
    N = K = 192  # x, dh and dx of one size
    gate, up, x = make(owq, N, K, 3, 5, M, M)
    rng = np.random.default_rng(M)
    dh = dev((0.01 * rng.standard_normal((M, N))).astype(np.float16))
    xd = dev(x)
    _, g, u = owq.gated(gate, up, xd, save=True)
    want = [host(t) for t in owq.gated_backward(gate, up, xd, g, u, dh)]
    (Lg, Lu), _ = owq._layers_on(("gate: ", gate), ("up: ", up))
    ws = torch.empty(owq.gated_backward_workspace_bytes(N, K, 3, 5, M), dtype=torch.uint8, device="cuda:0")
    for name in ("x", "g", "u", "dh"):
        print(f"dx over {name}: M={M}", flush=True)
        arrays = {"x": xd.clone(), "g": g.clone(), "u": u.clone(), "dh": dh.clone()}
        dw = [torch.zeros((N, k), device="cuda:0") for k in (3, 5)]
        st = owq.lib().owq_gated_backward(
            ctypes.byref(Lg), ctypes.byref(Lu), *[arrays[n].data_ptr() for n in ("x", "g", "u", "dh")], M, 0,
            arrays[name].data_ptr(), dw[0].data_ptr(), dw[1].data_ptr(), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert st == owq.OWQ_OK
        torch.cuda.synchronize()
        dx = host(arrays[name].view(torch.float16).reshape(-1)[:M * K].view(M, K))
        for a, b in zip((dx, host(dw[0]), host(dw[1])), want):
            assert a.tobytes() == b.tobytes(), name


def test_outputs_over_inputs_are_refused(owq):
    import torch
    N = K = 96
    gate, up, x = make(owq, N, K, 2, 2, 5, 1)
    xd = dev(x)
    with pytest.raises(owq.OwqError, match="RANGE.*overlaps x"):
        owq.gated(gate, up, xd, h=xd)
    ads = {"A": dev(np.ones((1, 4, K), np.float16)), "B": dev(np.ones((1, N, 4), np.float16)),
           "alpha": torch.ones(1, device="cuda:0")}
    which = torch.zeros(5, dtype=torch.int32, device="cuda:0")
    with pytest.raises(owq.OwqError, match="RANGE.*overlaps x"):
        owq.linear_adapters(gate, ads, which, xd, y=xd)
    t = torch.ones(10000, device="cuda:0")
    with pytest.raises(owq.OwqError, match="RANGE.*norm overlaps"):
        owq.clip_grad_norm([t], 1.0, norm=t[500:501])
    assert bool((t == 1.0).all())
