"""Low-rank adapters of many requests beside the packed linear
(owq_linear_adapters) on the GPU, against the definition in 64 bits.

Tolerance, per output: the shared product's bound of every linear test (2e-3
times its sum of absolute terms, plus 1e-5) is kept for the shared part. The
adapter part adds alpha sum_c B[i][c] t[c] with t an fp32 sum of exact products
(16 parts of K, each in steps of 32 products: chains of at most 32 + K / 512 + 16
roundings, relative 2^-16 of the absolute terms at K = 65536), kept in 22 bits of
the row's largest value, and an fp32 sum over at most 2 * 256 terms (2^-15); the
fp16 rounding of y (2^-11 of |y|) is the largest part of 2e-3. So the same 2e-3
holds with the absolute terms of the adapter part, alpha sum_c |B[i][c]| sum_j
|A[c][j] x[j]|, added to the bound."""
import numpy as np
import pytest

from mixed_precision_weight_amd import synth
from parity_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def _make(N, K, k, M, rank, count, seed):
    rng = np.random.default_rng(seed)
    W = synth.random_layer(rng, N, K, 0.02)
    idx = np.sort(rng.choice(K, k, replace=False)).astype(np.int32)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.choice(K, max(1, K // 200), replace=False)] *= 20.0
    A = (rng.standard_normal((count, rank, K)) / np.sqrt(K)).astype(np.float16)
    B = (0.1 * rng.standard_normal((count, N, rank))).astype(np.float16)
    alpha = (0.5 + 1.5 * rng.random(count)).astype(np.float32)
    return W, idx, x.astype(np.float16), A, B, alpha


def _reference(layer, x, A, B, alpha, which):
    """(y, bound) in 64 bits, from the packed layer as it stands."""
    import oracle
    ref = {"qcodes": host(layer["qcodes"]).view(np.uint32), "scales": host(layer["scales"]).view(np.uint16),
           "zeros": host(layer["zeros"]), "weak_idx": host(layer["weak_idx"]),
           "w_weak": host(layer["w_weak"]).view(np.uint16)}
    y, b = oracle.linear_rows(ref, x)
    y, b = np.array(y, np.float64), np.array(b, np.float64)
    x64 = x.astype(np.float64)
    for m, r in enumerate(which):
        if 0 <= r < len(alpha):
            t, ta = A[r].astype(np.float64) @ x64[m], np.abs(A[r].astype(np.float64)) @ np.abs(x64[m])
            y[m] += float(alpha[r]) * (B[r].astype(np.float64) @ t)
            b[m] += abs(float(alpha[r])) * (np.abs(B[r].astype(np.float64)) @ ta)
    return y, b


def _check(y, ref, bound, what):
    err = np.abs(host(y).astype(np.float64) - ref)
    assert (err <= 2e-3 * bound + 1e-5).all(), f"{what}: {np.max(err - 2e-3 * bound)}"


def _layer(owq, W, idx):
    return owq.pack(dev(W), dev(idx))


CASES = [
    # N, K, k, M, rank, count
    (1, 32, 0, 1, 1, 1),
    (17, 64, 3, 2, 5, 3),
    (130, 4096, 32, 1, 16, 8),
    (130, 4128, 7, 2, 64, 4),
    (67, 11008, 86, 1, 100, 3),
    (300, 768, 6, 3, 8, 5),
    (300, 768, 6, 4, 12, 5),
    (129, 1056, 9, 8, 16, 64),
    (200, 640, 0, 16, 33, 20),
    (513, 96, 96, 17, 4, 2),
    (200, 512, 5, 33, 256, 3),
    (257, 800, 9, 127, 16, 40),
    (260, 1024, 9, 128, 32, 7),
    (333, 992, 0, 300, 7, 130),
    (70, 65536, 9, 5, 3, 2),
    (190, 11008, 9, 40, 16, 3),
    (4200, 544, 9, 150, 8, 3),
    (20000, 96, 3, 260, 8, 3),
    (40000, 64, 3, 260, 4, 3),
    (44000, 64, 2, 40, 16, 3),
    (16600, 96, 3, 50, 12, 5),
    (22000, 160, 3, 200, 3, 4),
]


@pytest.mark.parametrize("case", CASES)
def test_against_the_definition(owq, case):
    import torch
    N, K, k, M, rank, count = case
    W, idx, x, A, B, alpha = _make(*case, seed=sum(case))
    layer = _layer(owq, W, idx)
    rng = np.random.default_rng(1)
    ads = {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}
    base = host(owq.linear(layer, dev(x)))
    for name, which in (
            ("mixed", rng.integers(-1, count, M)),
            ("one", np.full(M, count - 1)),
            ("none", np.full(M, -1)),
            ("past the end", np.where(np.arange(M) % 2 == 0, count, np.iinfo(np.int32).max)),
            ("runs", np.arange(M) * (count + 1) // M - 1)):
        which = which.astype(np.int32)
        print(f"adapters: {case} {name}", flush=True)
        ws = torch.full((owq.linear_adapters_workspace_bytes(rank, M),), 0xff, dtype=torch.uint8, device="cuda:0")
        y = owq.linear_adapters(layer, ads, dev(which), dev(x), workspace=ws)  # a workspace of NaN patterns
        torch.cuda.synchronize()
        ref, bound = _reference(layer, x, A, B, alpha, which)
        _check(y, ref, bound, name)
        none = (which < 0) | (which >= count)
        if M <= 16:  # the linear's own kernels; above, the sums have another order
            assert host(y)[none].tobytes() == base[none].tobytes(), name


@pytest.mark.parametrize("M", [2, 16, 40, 200])
def test_requests_do_not_reach_each_other(owq, M):
    """Infinities and NaN in one adapter, and the other tokens' order, change nothing for a token."""
    import torch
    N, K, k, rank, count = 150, 416, 4, 16, 6
    W, idx, x, A, B, alpha = _make(N, K, k, M, rank, count, 3)
    layer = _layer(owq, W, idx)
    which = (np.arange(M) % (count + 1) - 1).astype(np.int32)
    ads = {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}
    y = host(owq.linear_adapters(layer, ads, dev(which), dev(x)))
    for arr, val in ((A, np.inf), (A, np.nan), (B, np.inf), (B, np.nan)):
        for bad in (0, 3):
            a2, b2 = A.copy(), B.copy()
            (a2 if arr is A else b2)[bad] = val
            z = host(owq.linear_adapters(layer, {"A": dev(a2), "B": dev(b2), "alpha": dev(alpha)}, dev(which), dev(x)))
            ok = which != bad
            assert z[ok].tobytes() == y[ok].tobytes()
            assert not np.isfinite(z[~ok].astype(np.float32)).any()
    a2 = alpha.copy()
    a2[1] = np.nan
    z = host(owq.linear_adapters(layer, {"A": dev(A), "B": dev(B), "alpha": dev(a2)}, dev(which), dev(x)))
    assert z[which != 1].tobytes() == y[which != 1].tobytes()
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale", [2.0 ** -14, 2.0 ** 10])
@pytest.mark.parametrize("M", [1, 6, 30, 130])
def test_small_and_large_products(owq, scale, M):
    """A x far below and above fp16's range: it is kept relative to the row's largest value."""
    N, K, k, rank, count = 64, 2048, 0, 24, 2
    W, idx, x, A, B, alpha = _make(N, K, k, M, rank, count, 9)
    A = (A.astype(np.float64) * scale * 16).astype(np.float16)
    B = (B.astype(np.float64) / max(scale, 2.0 ** -8)).astype(np.float16)
    alpha = (alpha / (scale * max(1 / scale, 1))).astype(np.float32)
    layer = _layer(owq, W, idx)
    which = (np.arange(M) % 2).astype(np.int32)
    y = owq.linear_adapters(layer, {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}, dev(which), dev(x))
    ref, bound = _reference(layer, x, A, B, alpha, which)
    assert np.isfinite(host(y).astype(np.float32)).all()
    _check(y, ref, bound, f"scale {scale}")


@pytest.mark.parametrize("decode", ["vector", "matrix"])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_every_decode_kernel(owq, decode, M, monkeypatch):
    monkeypatch.setenv("OWQ_DECODE", decode)
    for products in ("dot2", "mfma"):
        monkeypatch.setenv("OWQ_GEMV_PRODUCTS", products)
        W, idx, x, A, B, alpha = _make(131, 544, 5, M, 72, 3, M)
        layer = _layer(owq, W, idx)
        which = np.array([2, -1, 0, 2][:M], np.int32)
        y = owq.linear_adapters(layer, {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}, dev(which), dev(x))
        ref, bound = _reference(layer, x, A, B, alpha, which)
        _check(y, ref, bound, f"{decode} {products}")


@pytest.mark.parametrize("M", [17, 1023, 1024, 1025, 2100])
def test_tokens_of_many_requests(owq, M):
    """More tokens than are grouped at a time, adapters 256 apart (one bucket), one token or all of one request:
    a token's output is that of the same token on its own rows, wherever it stands."""
    N, K, k, rank, count = 37, 96, 2, 4, 600
    W, idx, x, A, B, alpha = _make(N, K, k, M, rank, count, M)
    layer = _layer(owq, W, idx)
    ads = {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}
    rng = np.random.default_rng(M)
    for name, which in (("any", rng.integers(-3, count + 3, M)),
                        ("one bucket", 7 + 256 * rng.integers(0, 3, M)),
                        ("descending", (M - 1 - np.arange(M)) % count),
                        ("a lone one", np.where(np.arange(M) == M - 1, 255, -1)),
                        ("all", np.full(M, 511))):
        which = which.astype(np.int32)
        print(f"adapters: {M} tokens, {name}", flush=True)
        y = host(owq.linear_adapters(layer, ads, dev(which), dev(x)))
        ref, bound = _reference(layer, x, A, B, alpha, which)
        err = np.abs(y.astype(np.float64) - ref)
        assert (err <= 2e-3 * bound + 1e-5).all(), name
        turn = rng.permutation(M)
        z = host(owq.linear_adapters(layer, ads, dev(which[turn]), dev(np.ascontiguousarray(x[turn]))))
        assert z.tobytes() == y[turn].tobytes(), name


def test_graph_and_other_stream(owq):
    """Captured and replayed with the requests' adapters changing between replays; another stream."""
    import torch
    W, idx, x, A, B, alpha = _make(300, 1024, 9, 9, 16, 5, 4)
    layer = _layer(owq, W, idx)
    ads = {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}
    xd, wd = dev(x), dev(np.zeros(9, np.int32))
    y = torch.zeros((9, 300), dtype=torch.float16, device="cuda:0")
    owq.linear_adapters(layer, ads, wd, xd)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        owq.linear_adapters(layer, ads, wd, xd, y=y)
    for rep in range(3):
        which = ((np.arange(9) * (rep + 1)) % 6 - 1).astype(np.int32)
        wd.copy_(dev(which))
        g.replay()
        torch.cuda.synchronize()
        again = owq.linear_adapters(layer, ads, wd, xd)
        assert host(y).tobytes() == host(again).tobytes()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = owq.linear_adapters(layer, ads, wd, xd, stream=side)
    side.synchronize()
    assert host(z).tobytes() == host(y).tobytes()


def test_refusals_on_the_gpu(owq):
    import torch
    W, idx, x, A, B, alpha = _make(40, 64, 2, 3, 4, 2, 1)
    layer = _layer(owq, W, idx)
    ads = {"A": dev(A), "B": dev(B), "alpha": dev(alpha)}
    which = torch.zeros(3, dtype=torch.int32, device="cuda:0")
    with pytest.raises(owq.OwqError, match="WORKSPACE"):
        owq.linear_adapters(layer, ads, which, dev(x), workspace=torch.zeros(16, dtype=torch.uint8, device="cuda:0"))
    with pytest.raises(TypeError, match="CUDA"):
        owq.linear_adapters(layer, ads, which.cpu(), dev(x))
    off = torch.zeros(A.size + 1, dtype=torch.float16, device="cuda:0")[1:].view(2, 4, 64)
    with pytest.raises(owq.OwqError, match="ALIGN"):
        owq.linear_adapters(layer, {**ads, "A": off}, which, dev(x))
