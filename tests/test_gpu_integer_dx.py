"""dx of the integer form's backward in the bits that fp32 products would keep: one
rounding to fp16, and no row of the layer lost, over the forms' borders and long layers."""
import pytest
import torch

from integer_dx_util import faults
from integer_util import DEV, gen, tokens, weak_of, weights

pytestmark = pytest.mark.gpu


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


def _check(N, K, k, M, change=None):
    owq = _owq()
    g = gen(N + 3 * K + 5 * k + 7 * M)
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    dy = (torch.randn(M, N, generator=g, device=DEV) * 0.01).half()
    if change:
        change(g, L, dy)
    dx, _ = owq.linear_integer_backward(L, x, dy)
    found = faults(L["codes"], L["scales"], L["w_weak"], idx, dy, dx)
    assert not found, found


@pytest.mark.parametrize("M", [1, 31, 128, 129, 300])
@pytest.mark.parametrize("N,K,k", [(64, 96, 1), (513, 1056, 9), (768, 768, 6), (2731, 160, 40), (130, 4128, 33), (255, 256, 0),
                                   (257, 256, 0), (8200, 96, 6), (11008, 512, 32)])
def test_one_rounding(N, K, k, M):
    _check(N, K, k, M)


@pytest.mark.parametrize("N,K,k,M", [(4096, 4096, 32, 1000), (11008, 4096, 32, 2048)])
def test_one_rounding_of_whole_layers(N, K, k, M):
    _check(N, K, k, M)


def test_rows_and_tokens_of_very_different_size():
    def change(g, L, dy):
        L["scales"] *= 2.0 ** torch.randint(-6, 7, L["scales"].shape, generator=g, device=DEV).float()
        dy *= 2.0 ** torch.randint(-6, 7, (dy.shape[0], 1), generator=g, device=DEV).half()
        dy[3] = 0
        dy[4, 7] = 1000.0              # one gradient far above the others of its token
    _check(11008, 512, 32, 257, change)
    _check(1030, 320, 9, 40, change)
