"""The check of dx catches what it is for: a lost row, gradients in eleven bits, a lost part
of the contraction, and lets the 32-bit product pass."""
import pytest
import torch

from integer_dx_util import faults

# every layer of the GPU tests of dx (two of them with fewer columns), with few and more tokens
SIZES = [(N, K, k, M) for N, K, k in [(64, 96, 1), (513, 1056, 9), (768, 768, 6), (2731, 160, 40), (130, 4128, 33), (255, 256, 0),
                                      (257, 256, 0), (8200, 96, 6), (11008, 512, 32), (4096, 256, 32), (1030, 320, 9)]
         for M in (1, 31, 129)]


def _case(N, K, k, M):
    g = torch.Generator().manual_seed(N + K + k + M)
    codes = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8)
    codes = (codes.float() * torch.rand(N, K, generator=g)).round().to(torch.int8)
    idx = torch.sort(torch.randperm(K, generator=g)[:k]).values.to(torch.int32)
    codes[:, idx.long()] = 0
    scales = 0.0004 + 0.0003 * torch.rand(N, generator=g)
    w = (torch.randn(N, k, generator=g) * 0.02).half()
    dy = (torch.randn(M, N, generator=g) * 0.01).half()
    dy[:, -1] = 0.01                  # (the row that is lost below has gradients of the usual size)
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
    if M == 1:
        return
    zero = c[4].clone()
    zero[1] = 0                       # a token of zeros hides none of it
    c = c[:4] + (zero,)
    assert faults(*c, _dx(*c)) == []
    assert faults(*c, _dx(*c, rows=N - 1))
