"""A grid's threads are counted in 32 bits per dimension: sizes whose launches would
hold more are refused (OWQ_ERR_SHAPE) before anything is enqueued. CPU tests: every
call here is one that is refused before any HIP call; its pointers are not read."""
import ctypes

import pytest

SHAPE = 2


def AT(i):
    """Addresses that no array of these calls reaches from one to the next."""
    return (i + 1) << 52


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_weight_amd import owq
    return owq.lib()


def _layer(N, K=32, k=0):
    from mixed_precision_weight_amd.owq import OwqLayer
    return OwqLayer(N, K, k, 3, *[AT(i) for i in range(5)])


@pytest.mark.parametrize("N, M", [(2 ** 27, 1), (2 ** 27, 2), (2 ** 30, 1), (2 ** 30, 3), (2 ** 30, 16),
                                  (2 ** 30, 2 ** 10), (2 ** 19, 2 ** 19), (2 ** 26, 2 ** 24)])
def test_gated(lib, N, M):
    a = ctypes.byref(_layer(N))
    assert lib.owq_gated(a, a, AT(5), M, 0, AT(6), None, None, None) == SHAPE
    assert b"2^32" in lib.owq_last_error()


@pytest.mark.parametrize("M, k, want", [(2 ** 20, 512, "dx"), (2 ** 14, 32768, "dx"), (2 ** 20, 2048, "dw"),
                                        (2 ** 16, 32768, "dw"), (2 ** 20, 2048, "both")])
def test_gated_backward(lib, M, k, want):
    K = 32768
    a, b = _layer(64, K, k), _layer(64, K, k)
    need = lib.owq_gated_backward_workspace_bytes(64, K, k, k, M)
    assert need > 0
    dx = AT(9) if want != "dw" else None
    dwg, dwu = (AT(10), AT(11)) if want != "dx" else (None, None)
    assert lib.owq_gated_backward(ctypes.byref(a), ctypes.byref(b), AT(5), AT(6), AT(7), AT(8), M, 0, dx, dwg, dwu, AT(12),
                                  need, None) == SHAPE
    assert b"2^32" in lib.owq_last_error()


def _adapters(lib, N, M, rank):
    from mixed_precision_weight_amd.owq import OwqAdapters
    ad = OwqAdapters(AT(5), AT(6), AT(7), 3, rank)
    return lib.owq_linear_adapters(ctypes.byref(_layer(N)), ctypes.byref(ad), AT(8), AT(9), M, AT(10), AT(11), 2 ** 62,
                                   None)


@pytest.mark.parametrize("N, M, rank", [(64, 2 ** 21, 256), (64, 2 ** 25, 16), (64, 2 ** 25, 1), (64, 2 ** 30, 8),
                                        (201326593, 1, 8), (201326593, 2, 8), (2 ** 29, 4, 8), (2 ** 30, 16, 8),
                                        (2 ** 30, 2 ** 20, 8)])
def test_adapters(lib, N, M, rank):
    assert _adapters(lib, N, M, rank) == SHAPE
    assert b"2^32" in lib.owq_last_error()


def test_adapters_workspace(lib):
    f = lib.owq_linear_adapters_workspace_bytes
    for rank in (1, 16, 17, 100, 256):
        most = 2 ** 24 // ((rank + 15) // 16)  # the documented range
        assert f(rank, most) > 0
        assert f(rank, 2 * most) == 0


def test_clip_of_more_chunks_than_a_launch_counts(lib):
    from mixed_precision_weight_amd.owq import OwqGrad
    n = 2 ** 40
    items = (OwqGrad * 20)(*[OwqGrad(AT(i), AT(i), n, 0) for i in range(20)])
    need = lib.owq_clip_grad_norm_workspace_bytes(20)
    assert lib.owq_clip_grad_norm(items, 20, 1.0, AT(20), AT(21), need, None) == SHAPE
