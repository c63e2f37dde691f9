"""Outputs and workspaces of the block operators that lie over another array of the call
are refused (OWQ_ERR_RANGE): blocks that write them run beside blocks that still read.
CPU tests: refused before any HIP call; the pointers are not read."""
import ctypes

import pytest

RANGE = 3
N, K, k, M, rank, count = 64, 128, 4, 7, 16, 3


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_weight_amd import owq
    return owq.lib()


def _at(*names):
    """Addresses 1 MiB apart, more than any array of these calls has."""
    return {n: (i + 1) << 20 for i, n in enumerate(names)}


def _layer(at, tag, k=k):
    from mixed_precision_weight_amd.owq import OwqLayer
    return OwqLayer(N, K, k, 3, *[at[tag + n] for n in ("qcodes", "scales", "zeros", "weak_idx", "w_weak")])


LAYER = ("qcodes", "scales", "zeros", "weak_idx", "w_weak")
SIZE = {"qcodes": N * K // 8 * 3, "scales": 2 * N, "zeros": N, "weak_idx": 4 * k, "w_weak": 2 * N * k}


def _pairs(outs, ins, size, free=()):
    """(output, other, shift): the output moved so that it begins in, at or just before the other array."""
    for o in outs:
        for i in ins + outs:
            if i == o or (o, i) in free or (i, o) in free:
                continue
            align = 256 if "workspace" in (o, i) else 16
            inside = (size[i] - 1) // align * align
            for shift in sorted({0, inside, -((size[o] - 1) // align * align)}):
                yield o, i, shift


GATED_INS = ["x"] + ["g_" + n for n in LAYER] + ["u_" + n for n in LAYER]
GATED_SIZE = {"x": 2 * M * K, "h": 2 * M * N, "g": 4 * M * N, "u": 4 * M * N,
              **{t + n: s for t in ("g_", "u_") for n, s in SIZE.items()}}


@pytest.mark.parametrize("out, other, shift", _pairs(["h", "g", "u"], GATED_INS, GATED_SIZE))
def test_gated(lib, out, other, shift):
    at = _at("h", "g", "u", *GATED_INS)
    at[out] = at[other] + shift
    a, b = _layer(at, "g_"), _layer(at, "u_")
    assert lib.owq_gated(ctypes.byref(a), ctypes.byref(b), at["x"], M, 0, at["h"], at["g"], at["u"], None) == RANGE
    assert b"overlaps" in lib.owq_last_error()


BACK_INS = ["x", "g", "u", "dh"] + GATED_INS[1:]
BACK_OUTS = ["dx", "dw_gate", "dw_up", "workspace"]


def _back_sizes():
    from mixed_precision_weight_amd import owq
    return {**GATED_SIZE, "dh": 2 * M * N, "dx": 2 * M * K, "dw_gate": 4 * N * k, "dw_up": 4 * N * k,
            "workspace": owq.gated_backward_workspace_bytes(N, K, k, k, M)}


def test_gated_backward(lib):
    size = _back_sizes()
    assert max(size.values()) < 1 << 20
    for out, other, shift in _pairs(BACK_OUTS, BACK_INS, size, free=[("dx", n) for n in ("x", "g", "u", "dh")]):
        at = _at(*BACK_OUTS, *BACK_INS)
        at[out] = at[other] + shift
        a, b = _layer(at, "g_"), _layer(at, "u_")
        assert lib.owq_gated_backward(ctypes.byref(a), ctypes.byref(b), at["x"], at["g"], at["u"], at["dh"], M, 0, at["dx"],
                                      at["dw_gate"], at["dw_up"], at["workspace"], size["workspace"], None) == RANGE, (
            out, other, shift)
        assert b"overlaps" in lib.owq_last_error()


AD_INS = ["x", "A", "B", "alpha", "which"] + list(LAYER)


def test_adapters(lib):
    from mixed_precision_weight_amd import owq
    size = {**SIZE, "x": 2 * M * K, "A": 2 * count * rank * K, "B": 2 * count * N * rank, "alpha": 4 * count, "which": 4 * M,
            "y": 2 * M * N, "workspace": owq.linear_adapters_workspace_bytes(rank, M)}
    for out, other, shift in _pairs(["y", "workspace"], AD_INS, size):
        at = _at("y", "workspace", *AD_INS)
        at[out] = at[other] + shift
        L, ad = _layer(at, ""), owq.OwqAdapters(at["A"], at["B"], at["alpha"], count, rank)
        assert lib.owq_linear_adapters(ctypes.byref(L), ctypes.byref(ad), at["which"], at["x"], M, at["y"], at["workspace"],
                                       size["workspace"], None) == RANGE, (out, other, shift)
        assert b"overlaps" in lib.owq_last_error()


def test_clip(lib):
    from mixed_precision_weight_amd import owq
    size = {"norm": 4, "workspace": lib.owq_clip_grad_norm_workspace_bytes(2), "g0": 400, "g1": 100, "o1": 100}
    for out, other, shift in _pairs(["norm", "workspace"], ["g0", "g1", "o1"], size):
        at = _at(*size)
        at[out] = at[other] + shift
        items = (owq.OwqGrad * 2)(owq.OwqGrad(at["g0"], at["g0"], 100, 0), owq.OwqGrad(at["g1"], at["o1"], 50, 1))
        assert lib.owq_clip_grad_norm(items, 2, 1.0, at["norm"], at["workspace"], size["workspace"], None) == RANGE, (
            out, other, shift)
        assert b"overlaps" in lib.owq_last_error()
