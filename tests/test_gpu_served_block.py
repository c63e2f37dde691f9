"""The block operators together on the GPU, as a server and a tuner call them: an
adapted projection, the gated half and an adapted down projection one after another
(also captured, with the requests changing between replays), one layer given twice,
calls side by side on two streams, and workspaces used by one call after another.

Each stage is checked against 64 bits from the values that the stage before it
returned, with the tolerance of its own tests: the adapters' 2e-3 of the sum of
absolute terms plus 1e-5, the gated half's bound (test_gpu_gated)."""
import numpy as np
import pytest

import gated_util as gu
from mixed_precision_weight_amd import synth
from parity_util import dev, host
from test_gpu_gated import check as check_gated, reference as gated_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def owq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from mixed_precision_weight_amd import owq as o
    o.lib()
    return o


def _layer(owq, rng, N, K, k):
    W = synth.random_layer(rng, N, K, 0.6 / np.sqrt(K))
    return owq.pack(dev(W), dev(np.sort(rng.choice(K, k, replace=False)).astype(np.int32)))


def _adapters(rng, count, rank, N, K):
    a = {"A": (rng.standard_normal((count, rank, K)) / np.sqrt(K)).astype(np.float16),
         "B": (0.1 * rng.standard_normal((count, N, rank))).astype(np.float16),
         "alpha": (0.5 + rng.random(count)).astype(np.float32)}
    return a, {n: dev(v) for n, v in a.items()}


def _check_adapted(y, layer, a, which, x, what):
    W, x64 = gu.weights(layer), x.astype(np.float64)
    ref, bound = x64 @ W.T, np.abs(x64) @ np.abs(W).T
    for m, r in enumerate(which):
        if 0 <= r < len(a["alpha"]):
            A, B, al = a["A"][r].astype(np.float64), a["B"][r].astype(np.float64), float(a["alpha"][r])
            ref[m] += al * (B @ (A @ x64[m]))
            bound[m] += abs(al) * (np.abs(B) @ (np.abs(A) @ np.abs(x64[m])))
    err = np.abs(host(y).astype(np.float64) - ref)
    assert (err <= 2e-3 * bound + 1e-5).all(), what


@pytest.mark.parametrize("M", [1, 5, 16, 17, 90])
def test_block_of_many_requests(owq, M):
    import torch
    D, N, count = 288, 420, 5
    rng = np.random.default_rng(M)
    proj, gate, up, down = (_layer(owq, rng, D, D, 4), _layer(owq, rng, N, D, 5), _layer(owq, rng, N, D, 3),
                            _layer(owq, rng, D, 416, 6))
    a1, d1 = _adapters(rng, count, 8, D, D)
    a2, d2 = _adapters(rng, count, 12, D, 416)
    x = dev(rng.standard_normal((M, D)).astype(np.float16))
    which = dev(np.zeros(M, np.int32))
    # one workspace for both adapted projections: their calls are ordered
    ws = torch.empty(owq.linear_adapters_workspace_bytes(12, M), dtype=torch.uint8, device="cuda:0")

    def block(stream=None):
        y = owq.linear_adapters(proj, d1, which, x, workspace=ws, stream=stream)
        h = owq.gated(gate, up, y, act="silu", stream=stream)
        z = h[:, :416].contiguous()
        return y, h, z, owq.linear_adapters(down, d2, which, z, workspace=ws, stream=stream)

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block()
    for rep in range(4):
        requests = rng.integers(-1, count + 1, M).astype(np.int32)
        which.copy_(dev(requests))
        x.copy_(dev(rng.standard_normal((M, D)).astype(np.float16)))
        graph.replay()
        torch.cuda.synchronize()
        y, h, z, out = outs
        for a, b in zip(outs, block()):
            assert host(a).tobytes() == host(b).tobytes()
        _check_adapted(y, proj, a1, requests, host(x), "projection")
        check_gated(h, None, None, gated_reference(gate, up, host(y), "silu"), "gated")
        _check_adapted(out, down, a2, requests, host(z), "down projection")


@pytest.mark.parametrize("M", [1, 7, 60])
def test_one_layer_as_gate_and_up(owq, M):
    rng = np.random.default_rng(M)
    layer = _layer(owq, rng, 130, 256, 5)
    x = rng.standard_normal((M, 256)).astype(np.float16)
    h, g, u = owq.gated(layer, layer, dev(x), act="gelu", save=True)
    check_gated(h, g, u, gated_reference(layer, layer, x, "gelu"), "one layer")
    assert host(g).tobytes() == host(u).tobytes()
    dh = rng.standard_normal((M, 130)).astype(np.float16)
    dx, dwg, dwu = owq.gated_backward(layer, layer, dev(x), g, u, dev(dh), act="gelu")
    g64, u64, d64, W = (host(g).astype(np.float64), host(u).astype(np.float64), dh.astype(np.float64),
                        gu.weights(layer))
    value, slope = gu.act("gelu", g64)
    da, db = d64 * u64 * slope, d64 * value
    xw = x.astype(np.float64)[:, host(layer["weak_idx"])]
    # dx: A keeps 2^-11 of each term; dw: fp32 sums of exact products of da, db
    bound = np.abs(da) @ np.abs(W) + np.abs(db) @ np.abs(W)
    assert (np.abs(host(dx) - (da + db) @ W) <= 2.0 ** -9 * bound + 1e-6).all()
    for dw, d in ((dwg, da), (dwu, db)):
        assert (np.abs(host(dw) - d.T @ xw) <= 2.0 ** -14 * (np.abs(d).T @ np.abs(xw)) + 1e-7).all()


def test_calls_side_by_side(owq):
    """Two streams, each with its own workspaces and outputs, give what they give one after the other."""
    import torch
    rng = np.random.default_rng(5)
    M, N, K, count = 70, 300, 256, 4
    gate, up = _layer(owq, rng, N, K, 4), _layer(owq, rng, N, K, 4)
    _, ads = _adapters(rng, count, 16, N, K)
    runs = []
    for i in range(2):
        runs.append((dev(rng.standard_normal((M, K)).astype(np.float16)),
                     dev(rng.standard_normal((M, N)).astype(np.float16)),
                     dev(rng.integers(-1, count, M).astype(np.int32))))

    def work(run, stream=None):
        x, dh, which = run
        y = owq.linear_adapters(gate, ads, which, x, stream=stream)
        h, g, u = owq.gated(gate, up, x, save=True, stream=stream)
        dx, dwg, dwu = owq.gated_backward(gate, up, x, g, u, dh, stream=stream)
        norm = owq.clip_grad_norm([dwg, dwu], 0.1, stream=stream)
        return y, h, dx, dwg, dwu, norm

    want = [[host(t).copy() for t in work(run)] for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(work(runs[i], s))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for t, w in zip(outs, want[i]):
                assert host(t).tobytes() == w.tobytes()


@pytest.mark.parametrize("M", [1, 2, 4, 7, 16, 17, 70, 130])
def test_nothing_is_written_behind_the_ends(owq, M):
    """Outputs and workspaces of exactly the stated size, inside larger buffers whose other bytes stay as they were."""
    import torch
    N, K, count, rank = 131, 160, 3, 12
    rng = np.random.default_rng(M)
    gate, up = _layer(owq, rng, N, K, 4), _layer(owq, rng, N, K, 0)
    _, ads = _adapters(rng, count, rank, N, K)
    x = dev(rng.standard_normal((M, K)).astype(np.float16))
    dh = dev(rng.standard_normal((M, N)).astype(np.float16))
    which = dev(rng.integers(-1, count, M).astype(np.int32))
    guard, buffers = 4096, []

    def inside(shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((guard + n + guard,), 0xa5, dtype=torch.uint8, device="cuda:0")
        buffers.append((buf, n))
        return buf[guard:guard + n].view(dtype).view(shape)

    owq.linear_adapters(gate, ads, which, x, y=inside((M, N), torch.float16),
                        workspace=inside((owq.linear_adapters_workspace_bytes(rank, M),), torch.uint8))
    owq.gated(gate, up, x, h=inside((M, N), torch.float16))
    _, g, u = owq.gated(gate, up, x, save=True)
    dx, dwg, dwu = owq.gated_backward(gate, up, x, g, u, dh, workspace=inside(
        (owq.gated_backward_workspace_bytes(N, K, 4, 0, M),), torch.uint8))
    grads = [dwg, dx]
    outs = [inside(tuple(t.shape), t.dtype) for t in grads]
    owq.clip_grad_norm(grads, 1e-3, outs=outs,
                       workspace=inside((owq.clip_grad_norm_workspace_bytes([0, 0]),), torch.uint8))
    torch.cuda.synchronize()
    for i, (buf, n) in enumerate(buffers):
        assert int((buf[:guard] != 0xa5).sum()) == 0 and int((buf[guard + n:] != 0xa5).sum()) == 0, i


@pytest.mark.parametrize("M", [1, 3, 20, 100])
def test_arrays_at_any_element(owq, M):
    """Scales, weak weights, upstream gradients and outputs that start at an odd element give the same bits."""
    import torch
    N, K, count, rank = 96, 160, 3, 8
    rng = np.random.default_rng(M)
    gate, up = _layer(owq, rng, N, K, 9), _layer(owq, rng, N, K, 16)
    _, ads = _adapters(rng, count, rank, N, K)
    x = dev(rng.standard_normal((M, K)).astype(np.float16))
    dh = dev(rng.standard_normal((M, N)).astype(np.float16))
    which = dev(rng.integers(-1, count, M).astype(np.int32))

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:].copy_(t.reshape(-1))
        return buf[1:].view(t.shape)

    def run(gate, up, dh, h, y):
        owq.gated(gate, up, x, h=h)
        owq.linear_adapters(gate, ads, which, x, y=y)
        _, g, u = owq.gated(gate, up, x, save=True)
        return [host(t).tobytes() for t in (h, y) + tuple(owq.gated_backward(gate, up, x, g, u, dh))]

    out = torch.zeros((M, N), dtype=torch.float16, device="cuda:0")
    want = run(gate, up, dh, out, out.clone())
    moved = [{n: shifted(t) if t.dtype == torch.float16 else t for n, t in layer.items()} for layer in (gate, up)]
    assert moved[0]["scales"].data_ptr() % 4 == 2
    assert run(*moved, shifted(dh), shifted(out), shifted(out)) == want
