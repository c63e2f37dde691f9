"""The check of dx catches what it is for: a lost row, gradients in eleven bits, a lost part
of the contraction, and lets the 32-bit product pass."""
import pytest
import torch

from integer_dx_util import faults

SIZES = [(64, 96, 1, 31), (513, 256, 9, 40), (2731, 160, 40, 31), (130, 288, 33, 129), (8200, 64, 6, 33), (11008, 96, 32, 65)]


def _case(N, K, k, M):
    g = torch.Generator().manual_seed(N + K + k + M)
    codes = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8)
    codes = (codes.float() * torch.rand(N, K, generator=g)).round().to(torch.int8)
    idx = torch.sort(torch.randperm(K, generator=g)[:k]).values.to(torch.int32)
    codes[:, idx.long()] = 0
    scales = 0.0004 + 0.0003 * torch.rand(N, generator=g)
    w = (torch.randn(N, k, generator=g) * 0.02).half()
    dy = (torch.randn(M, N, generator=g) * 0.01).half()
    return codes, scales, w, idx, dy


def _dx(codes, scales, w, idx, dy, scaled=lambda g: g, rows=None):
    d = dy.float()
    g = scaled(d * scales[None, :])
    dx = g[:, :rows] @ codes.float()[:rows]
    dx[:, idx.long()] = d @ w.float()
    return dx.half()


def _eleven_bits(g):
    top = 2.0 ** torch.floor(torch.log2(g.abs().amax(1, keepdim=True)))
    return (g / top).half().float() * top


@pytest.mark.parametrize("N,K,k,M", SIZES)
def test_good_and_planted(N, K, k, M):
    c = _case(N, K, k, M)
    assert faults(*c, _dx(*c)) == []
    assert faults(*c, _dx(*c, rows=N - 1))
    assert faults(*c, _dx(*c, rows=N - 16))
    assert faults(*c, _dx(*c, scaled=_eleven_bits))
    zero = c[4].clone()
    zero[1] = 0                       # a token of zeros hides none of it
    c = c[:4] + (zero,)
    assert faults(*c, _dx(*c)) == []
    assert faults(*c, _dx(*c, rows=N - 1))
