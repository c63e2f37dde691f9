"""A layer in the storage-favoured form has codes of its dense columns only; with fewer
than 32 weak columns their shape is that of the per-row form. The entry points that take
the per-row form refuse it instead of reading its codes as other columns. CPU tests."""
import pytest
import torch

from mixed_precision_weight_amd import owq

N, K, M = 48, 128, 3


def _layer(k, storage):
    L = {"qcodes": torch.zeros((N, (K - k + 31) // 32 if storage else K // 32, 3), dtype=torch.int32),
         "scales": torch.zeros(N, dtype=torch.float16), "zeros": torch.zeros(N, dtype=torch.uint8),
         "w_weak": torch.zeros((N, k), dtype=torch.float16), "weak_idx": torch.arange(k, dtype=torch.int32)}
    return {**L, "K": K} if storage else L


def _calls():
    x, dh = torch.zeros((M, K), dtype=torch.float16), torch.zeros((M, N), dtype=torch.float16)
    g = torch.zeros((M, N))
    ads = {"A": torch.zeros((2, 4, K), dtype=torch.float16), "B": torch.zeros((2, N, 4), dtype=torch.float16),
           "alpha": torch.ones(2)}
    which = torch.zeros(M, dtype=torch.int32)
    ok = _layer(5, False)
    return {"gated, gate": lambda L: owq.gated(L, ok, x), "gated, up": lambda L: owq.gated(ok, L, x),
            "gated_backward": lambda L: owq.gated_backward(ok, L, x, g, g, dh),
            "linear_adapters": lambda L: owq.linear_adapters(L, ads, which, x),
            "linear": lambda L: owq.linear(L, x), "linear_backward": lambda L: owq.linear_backward(L, x, dh),
            "linear_batched": lambda L: owq.linear_batched([ok, L], [x, x])}


@pytest.mark.parametrize("call", sorted(_calls()))
def test_storage_form_is_refused(call):
    f = _calls()[call]
    with pytest.raises(ValueError, match="storage-favoured"):
        f(_layer(5, True))
    with pytest.raises(TypeError, match="CUDA"):  # all is well but for the device
        f(_layer(5, False))
    with pytest.raises(TypeError, match="CUDA"):  # without weak columns both forms are one
        f(_layer(0, True))


def test_fast_check_refuses_it_too():
    """The one-pass check that the calls on a GPU take first."""
    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0
    for storage in (False, True):
        L = {n: t.as_subclass(OnGpu) if isinstance(t, torch.Tensor) else t for n, t in _layer(5, storage).items()}
        assert (owq._layer_fast(L) is None) == storage
