"""The global gradient norm and clipping (owq_clip_grad_norm) on the GPU, against
numpy in 64 bits.

Tolerances. The norm's squares and sums are fp64 (relative error below 2^-40 for
the sizes here), so the fp32 norm is the rounded true value up to one tie:
relative 2^-24 plus 2^-40, taken as 2^-23. A clipped value is g * c with c in
fp64 (relative error below 2^-38), rounded once: half a step of its type,
relative 2^-24 (fp32) or 2^-11 (fp16), plus half of the type's smallest
subnormal; 2^-38 on top."""
import math

import numpy as np
import pytest

from parity_util import dev, host

pytestmark = pytest.mark.gpu

EPS = {np.float32: 2.0 ** -24, np.float16: 2.0 ** -11}
TINY = {np.float32: 2.0 ** -150, np.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def _grads(sizes, types, seed=0, sigma=0.01):
    rng = np.random.default_rng(seed)
    return [(rng.standard_normal(n) * sigma).astype(t) for n, t in zip(sizes, types)]


def _norm(gs):
    return math.sqrt(math.fsum(float(np.dot(g.astype(np.float64).ravel(), g.astype(np.float64).ravel())) for g in gs))


def _check(got, gs, max_norm, norm):
    want = _norm(gs)
    assert abs(float(host(norm)[0]) - want) <= 2.0 ** -23 * want, (float(host(norm)[0]), want)
    c = max_norm / want if want > max_norm else 1.0
    for i, (o, g) in enumerate(zip(got, gs)):
        t = g.dtype.type
        o = host(o)
        assert o.dtype == g.dtype and o.shape == g.shape
        if c == 1.0:
            assert o.tobytes() == g.tobytes(), i
            continue
        w = g.astype(np.float64) * c
        err = np.abs(o.astype(np.float64) - w)
        assert (err <= np.abs(w) * (EPS[t] + 2.0 ** -38) + TINY[t]).all(), (i, err.max())


CASES = [
    # sizes, types
    ([1], [np.float32]),
    ([1, 1], [np.float16, np.float32]),
    ([8191, 8192, 8193], [np.float32] * 3),
    ([8192, 0, 16384, 5, 0], [np.float16, np.float32, np.float16, np.float32, np.float16]),
    ([0, 0, 7], [np.float32] * 3),
    ([4096 * 32, 11008 * 32, 4096 * 86], [np.float32] * 3),
    ([3 * i * i % 20011 + 1 for i in range(301)], [np.float32 if i % 3 else np.float16 for i in range(301)]),
    ([7 + i for i in range(80)], [np.float16] * 80),
    ([7 + i for i in range(81)], [np.float32] * 81),
    ([5 + 40 * i for i in range(240)], [np.float32, np.float16] * 120),
    ([8193 - 30 * i for i in range(241)], [np.float16] * 241),
    ([0] * 240 + [9000, 0, 3], [np.float32] * 243),
    ([100 + i % 7 for i in range(483)], [np.float32] * 483),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("frac", [0.3, 1.7])
@pytest.mark.parametrize("inplace", [True, False])
def test_norm_and_clip(owq, case, frac, inplace):
    import torch
    sizes, types = CASES[case]
    gs = _grads(sizes, types, seed=case)
    print(f"clip: case {case}, {len(sizes)} tensors, {sum(sizes)} elements, limit {frac} of the norm", flush=True)
    limit = frac * _norm(gs)
    d = [dev(g) for g in gs]
    outs = None if inplace else [torch.full_like(t, 7.0) for t in d]
    norm = owq.clip_grad_norm(d, limit, outs=outs)
    torch.cuda.synchronize()
    _check(d if inplace else outs, gs, limit, norm)
    if not inplace:
        for t, g in zip(d, gs):
            assert host(t).tobytes() == g.tobytes()


def test_all_empty_and_zero_gradients(owq):
    import torch
    z = torch.zeros(0, device="cuda:0")
    assert float(owq.clip_grad_norm([z], 1.0)) == 0.0
    t = torch.zeros(10000, device="cuda:0")
    assert float(owq.clip_grad_norm([t, z], 0.0)) == 0.0
    assert int((t != 0).sum()) == 0


def test_zero_limit_and_no_limit(owq):
    import torch
    g = _grads([9000], [np.float32])[0]
    t = dev(g)
    owq.clip_grad_norm([t], math.inf)
    assert host(t).tobytes() == g.tobytes()
    o = torch.full_like(t, 3.0)
    owq.clip_grad_norm([t], math.inf, outs=[o])
    assert host(o).tobytes() == g.tobytes()
    owq.clip_grad_norm([t], 0.0)
    assert int((t != 0).sum()) == 0


def test_values_whose_squares_leave_fp32(owq):
    """Squares above and below fp32's range still count; a norm above it is infinite as fp32 and still clips."""
    big = np.full(5000, 1e30, np.float32)
    t = dev(big)
    norm = owq.clip_grad_norm([t], 1.0)
    _check([t], [big], 1.0, norm)
    small = np.full(5000, 1e-30, np.float32)
    t = dev(small)
    norm = owq.clip_grad_norm([t], 1e-29)
    _check([t], [small], 1e-29, norm)
    top = np.full(5000, 3e38, np.float32)
    t = dev(top)
    norm = owq.clip_grad_norm([t], 1e38)
    assert math.isinf(float(norm))
    w = 1e38 / math.sqrt(5000)
    assert abs(float(t[17]) - w) <= w * 2.0 ** -23


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_scales_nothing(owq, bad):
    gs = _grads([9000, 30], [np.float32, np.float16])
    gs[0][8999] = bad
    d = [dev(g) for g in gs]
    norm = float(owq.clip_grad_norm(d, 1e-3))
    assert not math.isfinite(norm)
    for t, g in zip(d, gs):
        assert host(t).tobytes() == g.tobytes()


def test_addresses_that_are_not_aligned(owq):
    """Views whose first element is at any multiple of the element size."""
    import torch
    for t, n in ((np.float32, 4), (np.float16, 8)):
        for off in range(n):
            g = _grads([20000], [t], seed=off)[0]
            buf = torch.zeros(20000 + 64, dtype=torch.float32 if t is np.float32 else torch.float16, device="cuda:0")
            v = buf[off:off + 20000]
            v.copy_(dev(g))
            limit = 0.5 * _norm([g])
            norm = owq.clip_grad_norm([v], limit)
            _check([v], [g], limit, norm)
            assert int((buf[:off] != 0).sum()) == 0 and int((buf[off + 20000:] != 0).sum()) == 0


def test_refusals(owq):
    import torch
    buf = torch.zeros(1000, device="cuda:0")
    with pytest.raises(owq.OwqError, match="RANGE.*twice"):
        owq.clip_grad_norm([buf, buf], 1.0)
    with pytest.raises(owq.OwqError, match="RANGE"):
        owq.clip_grad_norm([buf[:600], buf[500:]], 1.0)
    with pytest.raises(owq.OwqError, match="RANGE"):
        owq.clip_grad_norm([buf[:500]], 1.0, outs=[buf[100:600]])
    with pytest.raises(owq.OwqError, match="WORKSPACE"):
        owq.clip_grad_norm([buf], 1.0, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda:0"))
    # the same tensor read twice is two gradients
    o = [torch.zeros(1000, device="cuda:0") for _ in range(2)]
    buf.fill_(2.0)
    norm = owq.clip_grad_norm([buf, buf], math.inf, outs=o)
    assert abs(float(norm) - 2.0 * math.sqrt(2000)) <= 1e-4


def test_graph_and_other_stream(owq):
    """Captured and replayed, the limit met again each time, and run on a stream that is not the current one."""
    import torch
    gs = _grads([50000, 700, 8192], [np.float32, np.float16, np.float32], seed=5)
    limit = 0.25 * _norm(gs)
    src = [dev(g) for g in gs]
    d = [t.clone() for t in src]
    ws = torch.empty(owq.clip_grad_norm_workspace_bytes([1] * 3), dtype=torch.uint8, device="cuda:0")
    norm = torch.zeros(1, device="cuda:0")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        owq.clip_grad_norm(d, limit, norm=norm, workspace=ws)
    for rep in range(3):
        for t, s in zip(d, src):
            t.copy_(s * (1 if t.dtype == torch.float16 else 2 ** rep))
        now = [host(t).copy() for t in d]
        g.replay()
        torch.cuda.synchronize()
        _check(d, now, limit, norm)
    side = torch.cuda.Stream()
    d = [t.clone() for t in src]
    side.wait_stream(torch.cuda.current_stream())
    norm = owq.clip_grad_norm(d, limit, stream=side)
    side.synchronize()
    _check(d, gs, limit, norm)
