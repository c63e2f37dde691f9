"""What the integer form's entry points and the orthogonalised update refuse, in C and in
the binding. CPU tests: refused before any HIP call; the pointers are not read."""
import ctypes

import pytest
import torch

from mixed_precision_weight_amd import owq

NULL, SHAPE, RANGE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6
N, K, k, M = 64, 128, 4, 40


@pytest.fixture(scope="module")
def lib():
    return owq.lib()


def _at(*names):
    return {n: (i + 1) << 24 for i, n in enumerate(names)}


PARTS = ("codes", "scales", "weak_idx", "w_weak")
SIZE = {"codes": N * K, "scales": 4 * N, "weak_idx": 4 * k, "w_weak": 2 * N * k, "W": 2 * N * K, "x": 2 * M * K,
        "y": 2 * M * N, "dy": 2 * M * N, "dx": 2 * M * K, "dw": 4 * N * k}


def _layer(at, **kw):
    v = dict(N=N, K=K, k=k, **{n: at[n] for n in PARTS})
    v.update(kw)
    return owq.OwqIntegerLayer(*[v[f] for f, _ in owq.OwqIntegerLayer._fields_])


def _linear(lib, at, M=M, L=None, ws=1 << 20):
    L = L or _layer(at)
    return lib.owq_linear_integer(ctypes.byref(L), at["x"], M, at["y"], at["ws"], ws, None)


def _backward(lib, at, M=M, L=None, ws=1 << 23):
    L = L or _layer(at)
    return lib.owq_linear_integer_backward(ctypes.byref(L), at["x"], at["dy"], M, at["dx"], at["dw"], at["ws"], ws, None)


def _pack(lib, at, N=N, K=K, k=k):
    return lib.owq_pack_integer(at["W"], N, K, at["weak_idx"], k, at["codes"], at["scales"], at["w_weak"], None)


NAMES = PARTS + ("W", "x", "y", "dy", "dx", "dw", "ws")


@pytest.mark.parametrize("call", [_linear, _backward])
def test_layers_and_sizes(lib, call):
    at = _at(*NAMES)
    for kw, want in [({"N": 0}, SHAPE), ({"N": (1 << 30) + 1}, SHAPE), ({"K": 0}, SHAPE), ({"K": 33}, SHAPE),
                     ({"K": 65568}, SHAPE), ({"k": -1}, RANGE), ({"k": K + 1}, RANGE), ({"codes": None}, NULL),
                     ({"scales": None}, NULL), ({"weak_idx": None}, NULL), ({"w_weak": None}, NULL),
                     ({"codes": at["codes"] + 8}, ALIGN), ({"scales": at["scales"] + 2}, ALIGN),
                     ({"weak_idx": at["weak_idx"] + 2}, ALIGN), ({"w_weak": at["w_weak"] + 1}, ALIGN)]:
        assert call(lib, at, L=_layer(at, **kw)) == want, kw
    for m, want in [(0, SHAPE), (-1, SHAPE), ((1 << 30) + 1, SHAPE), (1 << 24, SHAPE)]:
        assert call(lib, at, M=m) == want, m
    assert call(lib, at, ws=255) == WORKSPACE
    for name, step in [("ws", 128), ("x", 8)]:
        assert call(lib, {**at, name: at[name] + step}) == ALIGN, name
    assert call(lib, {**at, "x": None}) == NULL
    assert call(lib, {**at, "ws": None}) == NULL


def test_tokens_that_a_launch_cannot_count(lib):
    at = _at(*NAMES)
    big = _layer(at, N=1 << 29)
    assert _linear(lib, at, M=1, L=big) == SHAPE
    assert _linear(lib, at, M=16, L=big) == SHAPE
    assert lib.owq_linear_integer_workspace_bytes(1 << 29, K, k, 16) == 0
    assert lib.owq_linear_integer_workspace_bytes(N, K, k, 1 << 24) == 0
    assert _pack(lib, at, N=1 << 24) == SHAPE
    assert _backward(lib, at, M=(1 << 20) + 1) == SHAPE
    assert lib.owq_linear_integer_backward_workspace_bytes(N, K, k, (1 << 20) + 1) == 0
    assert lib.owq_linear_integer_backward_workspace_bytes((1 << 20) + 1, K, k, 1) == 0


def test_workspaces(lib):
    assert lib.owq_linear_integer_workspace_bytes(N, K, k, 5) > 0
    for bad in [(0, K, k, M), (N, 0, k, M), (N, 40, k, M), (N, 65568, k, M), (N, K, -1, M), (N, K, K + 1, M), (N, K, k, 0)]:
        assert lib.owq_linear_integer_workspace_bytes(*bad) == 0
        assert lib.owq_linear_integer_backward_workspace_bytes(*bad) == 0
    at = _at(*NAMES)
    Ls = (owq.OwqIntegerLayer * 2)(_layer(at), _layer(at, N=7))
    one, two = (lib.owq_linear_integer_workspace_bytes(n, K, k, 16) for n in (N, 7))
    assert lib.owq_linear_integer_batched_workspace_bytes(Ls, 2, 16) == one + two
    for count, m in [(0, 16), (65, 16), (2, 0), (2, 17)]:
        assert lib.owq_linear_integer_batched_workspace_bytes(Ls, count, m) == 0


def test_pack(lib):
    at = _at(*NAMES)
    for kw, want in [({"N": 0}, SHAPE), ({"K": 48}, SHAPE), ({"k": -1}, RANGE), ({"k": K + 1}, RANGE)]:
        assert _pack(lib, at, **kw) == want, kw
    for n in ("W", "codes", "scales", "w_weak", "weak_idx"):
        assert _pack(lib, {**at, n: None}) == NULL, n
        assert _pack(lib, {**at, n: at[n] + 1}) == ALIGN, n


def _overlaps(outs, ins):
    for o in outs:
        for i in ins + outs:
            if i != o:
                for shift in (0, (SIZE.get(i, 256) - 1) // 256 * 256):
                    yield o, i, shift


@pytest.mark.parametrize("out,other,shift", _overlaps(["codes", "scales", "w_weak"], ["W", "weak_idx"]))
def test_pack_overlaps(lib, out, other, shift):
    at = _at(*NAMES)
    at[out] = at[other] + shift
    assert _pack(lib, at) == RANGE


@pytest.mark.parametrize("out,other,shift", _overlaps(["y", "ws"], ["x"] + list(PARTS)))
def test_linear_overlaps(lib, out, other, shift):
    at = _at(*NAMES)
    at[out] = at[other] + shift
    assert _linear(lib, at) == RANGE


@pytest.mark.parametrize("out,other,shift", _overlaps(["dx", "dw", "ws"], ["x", "dy"] + list(PARTS)))
def test_backward_overlaps(lib, out, other, shift):
    at = _at(*NAMES)
    at[out] = at[other] + shift
    assert _backward(lib, at) == RANGE


def _batched(lib, at, tags, M=16, count=None, ws=1 << 20):
    n = len(tags)
    P = ctypes.c_void_p * n
    Ls = (owq.OwqIntegerLayer * n)(*[_layer({p: at[t + p] for p in PARTS}) for t in tags])
    return lib.owq_linear_integer_batched(Ls, P(*[at[t + "x"] for t in tags]), P(*[at[t + "y"] for t in tags]),
                                          n if count is None else count, M, at["ws"], ws, None)


def test_batched(lib):
    at = _at("ws", *[t + n for t in "ab" for n in PARTS + ("x", "y")])
    for count, m, want in [(0, 16, UNSUPPORTED), (65, 16, UNSUPPORTED), (2, 0, UNSUPPORTED), (2, 17, UNSUPPORTED)]:
        assert _batched(lib, at, "ab", M=m, count=count) == want
    assert _batched(lib, at, "ab", ws=1024) == WORKSPACE
    for other in ["a" + n for n in PARTS + ("x", "y")] + ["ws"]:
        assert _batched(lib, {**at, "by": at[other]}, "ab") == RANGE, other
    assert _batched(lib, {**at, "bx": at["bx"] + 2}, "ab") == ALIGN
    assert b"layer 1" in lib.owq_last_error()


# ------------------------------------------------------------------ the update

COEF = (ctypes.c_double * 3)(3.4445, -4.7750, 2.0315)


def _ortho(lib, items, steps=5, coef=COEF, eps=1e-7, ws=1 << 40, wsb=1 << 30):
    arr = (owq.OwqUpdate * max(len(items), 1))(*[owq.OwqUpdate(*i) for i in items])
    return lib.owq_orthogonalize(arr, len(items), steps, coef, eps, ws, wsb, None)


G, O = 1 << 24, 1 << 28
ONE = (G, O, 300, 20, 1.0, 0)


def test_update_arguments(lib):
    for steps in (0, -1, 17):
        assert _ortho(lib, [ONE], steps=steps) == RANGE
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert _ortho(lib, [ONE], eps=eps) == RANGE
    for i in range(3):
        for bad in (float("inf"), float("nan")):
            c = [1.0, 1.0, 1.0]
            c[i] = bad
            assert _ortho(lib, [ONE], coef=(ctypes.c_double * 3)(*c)) == RANGE
    assert _ortho(lib, [ONE], coef=None) == NULL
    assert _ortho(lib, [ONE], ws=None) == NULL
    assert _ortho(lib, [ONE], ws=(1 << 40) + 64) == ALIGN
    assert _ortho(lib, [ONE], wsb=100) == WORKSPACE
    assert _ortho(lib, []) == UNSUPPORTED
    for item, want in [((G, O, -1, 20, 1.0, 0), SHAPE), ((G, O, 20, -1, 1.0, 0), SHAPE), ((G, O, (1 << 20) + 1, 2, 1.0, 0), SHAPE),
                       ((G, O, 16385, 16385, 1.0, 0), SHAPE), ((G, O, 300, 20, float("inf"), 0), RANGE),
                       ((G, O, 300, 20, float("nan"), 0), RANGE), ((G, O, 300, 20, 1.0, 2), UNSUPPORTED),
                       ((G, O, 300, 20, 1.0, -1), UNSUPPORTED), ((None, O, 300, 20, 1.0, 0), NULL),
                       ((G, None, 300, 20, 1.0, 0), NULL), ((G + 2, O, 300, 20, 1.0, 0), ALIGN),
                       ((G, O + 1, 300, 20, 1.0, 1), ALIGN)]:
        assert _ortho(lib, [item]) == want, item


def test_update_overlaps(lib):
    n = 300 * 20 * 4
    assert _ortho(lib, [(G, G + n - 4, 300, 20, 1.0, 0)]) == RANGE          # out begins inside g
    assert _ortho(lib, [ONE, ONE]) == RANGE                                 # the same out twice
    assert _ortho(lib, [ONE, (O + n - 256, O + n, 300, 20, 1.0, 0)]) == RANGE   # an out over another g
    assert _ortho(lib, [(G, G, 300, 20, 1.0, 0), (G + 4, O, 300, 20, 1.0, 0)]) == RANGE
    for at in (G, O, G + n // 256 * 256, O - 256):
        assert _ortho(lib, [ONE], ws=at) == RANGE, at


def test_update_workspace(lib):
    def need(*shapes):
        return owq.orthogonalize_workspace_bytes(list(shapes))
    assert need((300, 20)) > 0 and need((300, 200)) > 4 * 300 * 200
    assert need((0, 5)) > 0
    for bad in [(-1, 5), (5, -1), ((1 << 20) + 1, 1), (16385, 20000)]:
        assert need(bad) == 0
    assert lib.owq_orthogonalize_workspace_bytes(None, 1) == 0
    assert need() == 0


# -------------------------------------------------------------------- the binding


def _cpu_layer(N=8, K=64, k=2):
    return {"codes": torch.zeros(N, K, dtype=torch.int8), "scales": torch.zeros(N), "w_weak": torch.zeros(N, k).half(),
            "weak_idx": torch.arange(k, dtype=torch.int32)}


def test_binding_checks_shapes_before_devices():
    L = _cpu_layer()
    x = torch.zeros(3, 64).half()
    with pytest.raises(ValueError, match="columns"):
        owq.linear_integer(L, torch.zeros(3, 32).half())
    with pytest.raises(TypeError, match="float16"):
        owq.linear_integer(L, torch.zeros(3, 64))
    with pytest.raises(ValueError, match="contiguous"):
        owq.linear_integer(L, torch.zeros(64, 3).half().t())
    with pytest.raises(ValueError, match="expected"):
        owq.linear_integer(L, x, y=torch.zeros(3, 9).half())
    for name in L:
        short = {n: t for n, t in L.items() if n != name}
        with pytest.raises(ValueError, match=name):
            owq.linear_integer(short, x)
    for name, t in [("codes", L["codes"].to(torch.uint8)), ("scales", L["scales"].half()), ("scales", torch.zeros(9)),
                    ("w_weak", torch.zeros(8, 3).half()), ("weak_idx", L["weak_idx"].long())]:
        with pytest.raises((TypeError, ValueError), match=name):
            owq.linear_integer({**L, name: t}, x)
    with pytest.raises(TypeError, match="CUDA"):
        owq.linear_integer(L, x)
    with pytest.raises(ValueError, match="qcodes|codes"):
        owq.linear_integer({"qcodes": torch.zeros(8, 2, 3, dtype=torch.int32)}, x)
    with pytest.raises(ValueError, match="dy has shape"):
        owq.linear_integer_backward(L, x, torch.zeros(3, 9).half())
    with pytest.raises(ValueError, match="as many x"):
        owq.linear_integer_batched([L, L], [x])
    with pytest.raises(ValueError, match="rows"):
        owq.linear_integer_batched([L, L], [x, torch.zeros(2, 64).half()])
    with pytest.raises(ValueError, match="multiple of 32"):
        owq.pack_integer(torch.zeros(4, 40).half(), torch.arange(2, dtype=torch.int32))


def test_binding_of_the_update():
    m = torch.zeros(4, 3)
    with pytest.raises(ValueError, match="1 to 4096"):
        owq.orthogonalize([])
    with pytest.raises(TypeError, match="float32 or torch.float16"):
        owq.orthogonalize([m.double()])
    with pytest.raises(ValueError, match="2-D"):
        owq.orthogonalize([torch.zeros(4)])
    with pytest.raises(ValueError, match="contiguous"):
        owq.orthogonalize([torch.zeros(4, 3).t()])
    with pytest.raises(ValueError, match="one out"):
        owq.orthogonalize([m], outs=[m, m])
    with pytest.raises(ValueError, match="one scale"):
        owq.orthogonalize([m], scales=[])
    with pytest.raises(ValueError, match="shape"):
        owq.orthogonalize([m], outs=[torch.zeros(3, 4)])
    with pytest.raises(TypeError, match="out"):
        owq.orthogonalize([m], outs=[m.half()])
    with pytest.raises(ValueError, match="three"):
        owq.orthogonalize([m], coefficients=(1.0, 2.0))
    with pytest.raises(TypeError, match="CUDA"):
        owq.orthogonalize([m])
