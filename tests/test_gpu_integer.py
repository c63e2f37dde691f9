"""The integer form's pack and product against the definition in 64 bits, over the
forms' borders (tokens 4 | 5, 16 | 17, 32 | 33, 64 | 65, 256 | 257), odd and ragged sizes, no weak
column, every column weak, zero rows, non-finite tokens, streams, graphs."""
import pytest
import torch

from integer_util import (DEV, check_product, gen, rows_quantised, tokens, weak_of, weights)

pytestmark = pytest.mark.gpu

SIZES = [(1, 32, 0), (1, 32, 32), (16, 64, 1), (200, 96, 7), (513, 1056, 9), (768, 768, 6), (40, 4128, 33),
         (300, 11008, 86), (1031, 4096, 32)]


def _owq():
    from mixed_precision_weight_amd import owq
    return owq


@pytest.mark.parametrize("N,K,k", SIZES + [(3, 65536, 5)])
def test_pack_is_the_definition(N, K, k):
    owq = _owq()
    g = gen(N * 7 + K + k)
    W, idx = weights(g, N, K), weak_of(g, K, k)
    W[0] = 0
    if N > 2:
        W[1] *= 300.0
        W[2] = (W[2].float() * 2.0 ** -12).half()   # subnormal values
    L = owq.pack_integer(W, idx)
    q, s = rows_quantised(W, idx)
    assert torch.equal(L["codes"].double(), q)
    assert torch.equal(L["scales"].double(), s)
    assert torch.equal(L["w_weak"], W[:, idx.long()])
    out = {n: torch.empty_like(L[n]) for n in ("codes", "scales", "w_weak")}
    assert owq.pack_integer(W, idx, out=out) is out
    assert torch.equal(out["codes"], L["codes"])


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 16, 17, 32, 33, 64, 65, 128, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K,k", SIZES)
def test_product(N, K, k, M):
    owq = _owq()
    g = gen(N + 3 * K + 5 * k + 7 * M)
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    if M > 2:
        x[1] = 0          # a token of zeros
    check_product(L, x, owq.linear_integer(L, x))


@pytest.mark.parametrize("M", [1, 16, 40])
def test_product_of_the_longest_rows(M):
    owq = _owq()
    g = gen(65536 + M)
    idx = weak_of(g, 65536, 40)
    L = owq.pack_integer(weights(g, 70, 65536), idx)
    x = tokens(g, M, 65536, idx)
    check_product(L, x, owq.linear_integer(L, x))
    # every code and every token at the ends of the range: the integer sum's largest value
    L["codes"].fill_(127)
    L["codes"][:, idx.long()] = 0
    x.fill_(-1.5)
    check_product(L, x, owq.linear_integer(L, x))


@pytest.mark.parametrize("M", [1, 9, 200])
def test_every_output_is_written_and_nothing_else(M):
    owq = _owq()
    g = gen(M)
    N, K, k = 333, 160, 5
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    room = torch.full((M * N + 64,), 7.0, dtype=torch.float16, device=DEV)
    y = room[32:32 + M * N].view(M, N)
    need = owq.linear_integer_workspace_bytes(N, K, k, M)
    ws = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device=DEV)
    off = (-ws.data_ptr()) % 256
    assert owq.linear_integer(L, x, y=y, workspace=ws[off:off + max(need, 1)]) is y
    check_product(L, x, y)
    assert bool((room[:32] == 7).all()) and bool((room[32 + M * N:] == 7).all())
    assert bool((ws[:off] == 0xa5).all()) and bool((ws[off + need:] == 0xa5).all())


@pytest.mark.parametrize("M", [2, 7, 40, 200])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_token_that_is_not_finite_stays_alone(M, bad):
    owq = _owq()
    g = gen(M)
    N, K, k = 130, 224, 6
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    good = owq.linear_integer(L, x)
    dense = next(j for j in range(K) if j not in idx.tolist())
    x[M - 1, dense] = bad
    y = owq.linear_integer(L, x)
    assert torch.equal(y[:M - 1], good[:M - 1])
    assert not bool(torch.isfinite(y[M - 1]).any())
    x[M - 1] = 0
    x[M - 1, int(idx[2])] = bad     # in a weak column it multiplies its weights alone
    y = owq.linear_integer(L, x)
    assert torch.equal(y[:M - 1], good[:M - 1])
    assert not bool(torch.isfinite(y[M - 1][L["w_weak"][:, 2] != 0]).any())


@pytest.mark.parametrize("M", [1, 3, 4, 5, 16])
def test_batched_is_bit_for_bit_the_single_call(M):
    owq = _owq()
    g = gen(100 + M)
    shapes = [(64, 96, 3), (700, 4096, 32), (17, 32, 0), (300, 1056, 9)] * 5   # more than one launch's layers
    layers, xs = [], []
    for N, K, k in shapes:
        idx = weak_of(g, K, k)
        layers.append(owq.pack_integer(weights(g, N, K), idx))
        xs.append(tokens(g, M, K, idx))
    ys = owq.linear_integer_batched(layers, xs)
    for L, x, y in zip(layers, xs, ys):
        assert torch.equal(y, owq.linear_integer(L, x))
        check_product(L, x, y)


@pytest.mark.parametrize("M", [1, 12, 77])
def test_other_stream_and_graph(M):
    owq = _owq()
    g = gen(200 + M)
    N, K, k = 515, 1056, 9
    idx = weak_of(g, K, k)
    L = owq.pack_integer(weights(g, N, K), idx)
    x = tokens(g, M, K, idx)
    want = owq.linear_integer(L, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = owq.linear_integer(L, x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = owq.linear_integer(L, x)
    for seed in range(3):
        x.copy_(tokens(gen(seed), M, K, idx))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, owq.linear_integer(L, x))
