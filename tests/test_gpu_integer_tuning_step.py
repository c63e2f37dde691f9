"""One step of weak-column tuning on a layer of the integer form, as a program runs it:
product, backward, clipping, orthogonalised update, new weak weights, product again."""
import math

import pytest
import torch

from integer_util import DEV, check_backward, check_orthogonal, check_product, gen, tokens, weak_of, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 40, 300])
def test_step(M):
    from mixed_precision_weight_amd import owq
    g = gen(M)
    shapes = [(513, 1056, 9), (1056, 512, 32), (200, 96, 0)]
    layers, xs, dys = [], [], []
    for N, K, k in shapes:
        idx = weak_of(g, K, k)
        layers.append(owq.pack_integer(weights(g, N, K), idx))
        xs.append(tokens(g, M, K, idx))
        dys.append((torch.randn(M, N, generator=g, device=DEV) * 0.01).half())
    ys = owq.linear_integer_batched(layers, xs) if M <= 16 else [owq.linear_integer(L, x) for L, x in zip(layers, xs)]
    grads = []
    for L, x, y, dy in zip(layers, xs, ys, dys):
        check_product(L, x, y)
        dx, dw = owq.linear_integer_backward(L, x, dy)
        check_backward(L, x, dy, dx, dw)
        grads.append(dw)
    before = [d.clone() for d in grads]
    norm = owq.clip_grad_norm(grads, 0.5)
    want = math.sqrt(sum(float((d.double() ** 2).sum()) for d in before))
    assert abs(float(norm) - want) <= 1e-6 * want
    clipped = [d.clone() for d in grads]
    steps = owq.orthogonalize(grads, scales=[0.02 * math.sqrt(max(1.0, N / max(k, 1))) for N, K, k in shapes])
    for (N, K, k), L, c, s, x in zip(shapes, layers, clipped, steps, xs):
        if k:
            check_orthogonal(c, s, 5, owq.NEWTON_SCHULZ, 1e-7, 0.02 * math.sqrt(max(1.0, N / k)))
        old = owq.linear_integer(L, x)
        L["w_weak"].copy_((L["w_weak"].float() - s).half())
        y = owq.linear_integer(L, x)
        check_product(L, x, y)
        assert k == 0 or not torch.equal(y, old)
