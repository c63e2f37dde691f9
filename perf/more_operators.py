"""The integer form of the mixed-precision linear and the orthogonalised update, as
they are measured.

Four kinds of call:

  linear   y = x W^T with W and every token in 8-bit integers (a scale per output
           channel and per token) and the weak columns in fp16 on both sides
  batched  several such linears on the same number of tokens in one call
  grad     its backward for weak-column tuning: dx and the weak columns' gradient
  ortho    many gradient matrices, each replaced by an orthogonal factor of itself
           (Newton-Schulz products), the update that follows the clipping

``run`` with ``own`` false is the plain form: the definitions in elementary torch
operations in 32 bits. With ``own`` true it makes the framework's calls. ``exact``
evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda:0"

# the odd quintic of the orthogonalisation, five products of each kind
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7

# the seven linears of a 7B decoder layer as (rows, columns, weak columns)
LAYER_7B = "4096x4096/32*4 11008x4096/32*2 4096x11008/86"

# ------------------------------------------------------------------- the cases


def listed():
    return [
        # one token through an attention projection of a small model: latency alone counts
        {"name": "linear_decode_1_small", "op": "linear", "M": 1, "K": 768, "N": 768, "k": 6},
        # one token of one user through the seven linears of a 7B decoder layer: the weights' bytes count
        {"name": "batched_decode_1_layer", "op": "batched", "M": 1, "layers": LAYER_7B},
        # one token each of sixteen users, gate projection of a 7B decoder layer
        {"name": "linear_decode_16", "op": "linear", "M": 16, "K": 4096, "N": 11008, "k": 32},
        # a short prompt on a small layer of uneven sizes
        {"name": "linear_ragged", "op": "linear", "M": 77, "K": 1056, "N": 2731, "k": 9},
        # a prompt of 300 tokens, down projection of a 7B decoder layer
        {"name": "linear_prompt_300", "op": "linear", "M": 300, "K": 11008, "N": 4096, "k": 86},
        # a prompt of 2048 tokens, gate projection of a 7B decoder layer: the products count
        {"name": "linear_prefill", "op": "linear", "M": 2048, "K": 4096, "N": 11008, "k": 32},
        # a short last batch of a tuning run on a small layer of uneven sizes
        {"name": "grad_ragged", "op": "grad", "M": 77, "K": 1056, "N": 2731, "k": 9},
        # a training step of weak-column tuning, one sequence of 2048 tokens, gate projection of a 7B layer
        {"name": "grad_train", "op": "grad", "M": 2048, "K": 4096, "N": 11008, "k": 32},
        # the weak columns' gradients of one 7B decoder layer
        {"name": "ortho_layer", "op": "ortho", "shapes": "4096x32*4 11008x32*2 4096x86", "type": "fp32"},
        # the weak columns' gradients of all 32 layers
        {"name": "ortho_model", "op": "ortho", "shapes": "4096x32*128 11008x32*64 4096x86*32", "type": "fp32"},
        # half-precision gradients: weak columns of two large layers, both factors of some low-rank adapters
        {"name": "ortho_mixed_half", "op": "ortho", "shapes": "28672x63*2 8192x221*2 64x4096*4 11008x64*4 16x4099*3",
         "type": "fp16"},
        # a matrix that is tuned whole
        {"name": "ortho_dense", "op": "ortho", "shapes": "4096x2048", "type": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["flops"] / 500e12 + w["bytes"] / 4e12


def draw(rng):
    op = rng.choice(["linear", "batched", "grad", "ortho"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "ortho":
            groups = []
            for _ in range(rng.randint(1, 3)):
                long, short = _log_int(rng, 1, 16384), _log_int(rng, 1, 1024)
                a, b = (long, short) if rng.random() < 0.7 else (short, long)
                groups.append(f"{a}x{b}*{_log_int(rng, 1, 40)}")
            case = {"op": op, "shapes": " ".join(groups), "type": rng.choice(["fp32", "fp16"])}
        elif op == "batched":
            groups = []
            for _ in range(rng.randint(1, 3)):
                K = 32 * _log_int(rng, 2, 344)
                k = min(K, rng.choice([0, 1, 6, 9, 32, 63, 86]))
                groups.append(f"{_log_int(rng, 40, 11008)}x{K}/{k}*{rng.randint(1, 4)}")
            case = {"op": op, "M": _log_int(rng, 1, 16), "layers": " ".join(groups)}
        else:
            K = 32 * _log_int(rng, 2, 344)
            case = {"op": op, "M": _log_int(rng, 1, 2048), "K": K, "N": _log_int(rng, 40, 28672),
                    "k": min(K, rng.choice([0, 1, 6, 9, 32, 63, 86]))}
        if _cost(case) <= most:
            return case


def _shapes(case):
    """[(rows, columns)] of an orthogonalisation."""
    out = []
    for part in case["shapes"].split():
        shape, _, times = part.partition("*")
        rows, cols = shape.split("x")
        out += [(int(rows), int(cols))] * int(times or 1)
    return out


def _layers(case):
    """[(N, K, k)] of a call on 8-bit layers."""
    if case["op"] != "batched":
        return [(case["N"], case["K"], case["k"])]
    out = []
    for part in case["layers"].split():
        layer, _, times = part.partition("*")
        shape, k = layer.split("/")
        N, K = shape.split("x")
        out += [(int(N), int(K), int(k))] * int(times or 1)
    return out


def work(case):
    if case["op"] == "ortho":
        size = 4 if case["type"] == "fp32" else 2
        bytes_, flops = 0, 0
        for r, c in _shapes(case):
            s = min(r, c)
            bytes_ += 2 * r * c * size
            # the Gram matrix (symmetric), the matrix times its polynomial, and the
            # polynomial's products of symmetric s x s matrices that commute
            flops += 3 * r * c * s + (4 * STEPS - 3) * s * s * s
        return {"bytes": bytes_, "flops": flops}
    M = case["M"]
    bytes_, flops = 0, 0
    for N, K, k in _layers(case):
        layer = N * K + 4 * N + 2 * N * k + 4 * k
        if case["op"] == "grad":
            # dy and the weak columns of x read, dx and the weak gradient written
            bytes_ += layer + 2 * M * N + 2 * M * k + 2 * M * K + 4 * N * k
            flops += 2 * M * N * K + 4 * M * N * k
        else:
            bytes_ += layer + 2 * M * K + 2 * M * N
            flops += 2 * M * N * K + 2 * M * N * k
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ the inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _layer(g, N, K, k):
    """An 8-bit layer of Gaussian weights: per row scale = max |w| / 127 over its
    dense columns, codes rint(w * (127 / max |w|)), 0 at the k weak columns."""
    W = (torch.randn(N, K, generator=g, device=DEV) * 0.02).half()
    idx = torch.sort(torch.randperm(K, generator=g, device=DEV)[:k]).values
    dense = W.float()
    dense[:, idx] = 0.0
    top = dense.abs().amax(1, keepdim=True)
    full = torch.full_like(top, 127.0)  # (of tensors, so that each is one division)
    codes = torch.round(dense * torch.where(top > 0, full / top, torch.zeros_like(top)))
    return {"codes": codes.to(torch.int8), "scales": (top / full).view(N).contiguous(),
            "w_weak": W[:, idx].contiguous(), "weak_idx": idx.to(torch.int32)}


def _activations(g, M, K, idx):
    """Layer input: unit Gaussian, the weak columns' channels twenty times as large."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, idx.long()] *= 20.0
    return x.half()


def _gradient(g, rows, cols):
    """A gradient matrix: a few strong directions over a Gaussian floor."""
    q = min(rows, cols, 8)
    strong = torch.randn(rows, q, generator=g, device=DEV) * (4.0 * 0.6 ** torch.arange(q, device=DEV))
    return 0.01 * (strong @ torch.randn(q, cols, generator=g, device=DEV)
                   + torch.randn(rows, cols, generator=g, device=DEV))


def _arena(shapes, dt):
    """One zeroed buffer and a matrix of each shape in it, each starting at a
    multiple of 64 elements (how a program keeps its updates)."""
    starts, end = [], 0
    for r, c in shapes:
        starts.append(end)
        end += (r * c + 63) // 64 * 64
    flat = torch.zeros(end, dtype=dt, device=DEV)
    return flat, [flat[b:b + r * c].view(r, c) for b, (r, c) in zip(starts, shapes)]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if own:
        from mixed_precision_weight_amd import owq
        s["owq"] = owq
    if case["op"] == "ortho":
        dt = torch.float32 if case["type"] == "fp32" else torch.float16
        shapes = _shapes(case)
        s["updates"] = [_gradient(g, r, c).to(dt) for r, c in shapes]
        s["scales"] = [math.sqrt(max(1.0, r / c)) for r, c in shapes]
        s["flat"], s["outs"] = _arena(shapes, dt)
        if own:
            s["workspace"] = torch.empty(owq.orthogonalize_workspace_bytes(shapes), dtype=torch.uint8, device=DEV)
        return s
    M, shapes = case["M"], _layers(case)
    s["layers"] = [_layer(g, N, K, k) for N, K, k in shapes]
    s["xs"] = [_activations(g, M, K, L["weak_idx"]) for (N, K, k), L in zip(shapes, s["layers"])]
    if case["op"] == "grad":
        s["dy"] = (torch.randn(M, case["N"], generator=g, device=DEV) * 0.01).half()
    if own:
        if case["op"] == "grad":
            need = owq.linear_integer_backward_workspace_bytes(case["N"], case["K"], case["k"], M)
        elif case["op"] == "batched":
            need = owq.linear_integer_batched_workspace_bytes(shapes, M)
        else:
            need = owq.linear_integer_workspace_bytes(case["N"], case["K"], case["k"], M)
        s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- the plain form


def _plain_linear(layer, x):
    x, idx = x.float(), layer["weak_idx"].long()
    weak = x[:, idx]
    dense = x.clone()
    dense[:, idx] = 0.0
    top = dense.abs().amax(1, keepdim=True)
    full = torch.full_like(top, 127.0)
    codes = torch.round(dense * torch.where(top > 0, full / top, torch.zeros_like(top)))
    y = (codes @ layer["codes"].float().t()) * (top / full) * layer["scales"][None, :]
    return (y + weak @ layer["w_weak"].float().t()).half()


def _plain(s):
    case = s["case"]
    if case["op"] == "ortho":
        a, b, c = COEFFICIENTS
        for u, o, scale in zip(s["updates"], s["outs"], s["scales"]):
            X = u.float()
            X = X / (X.pow(2).sum().sqrt() + EPS)
            wide = X.shape[0] <= X.shape[1]
            for _ in range(STEPS):
                A = X @ X.t() if wide else X.t() @ X
                B = b * A + c * (A @ A)
                X = a * X + (B @ X if wide else X @ B)
            o.copy_(scale * X)
        return s["flat"]
    if case["op"] == "grad":
        layer, dy = s["layers"][0], s["dy"].float()
        idx = layer["weak_idx"].long()
        dx = (dy * layer["scales"][None, :]) @ layer["codes"].float()
        dx[:, idx] = dy @ layer["w_weak"].float()
        return {"dx": dx.half(), "dw_weak": dy.t() @ s["xs"][0].float()[:, idx]}
    ys = [_plain_linear(L, x) for L, x in zip(s["layers"], s["xs"])]
    return ys if case["op"] == "batched" else ys[0]


# ---------------------------------------------------------------- one pass


def run(state):
    if not own:
        return _plain(state)
    s, owq = state, state["owq"]
    op = s["case"]["op"]
    if op == "ortho":
        owq.orthogonalize(s["updates"], outs=s["outs"], scales=s["scales"], steps=STEPS, coefficients=COEFFICIENTS,
                          eps=EPS, workspace=s["workspace"])
        return s["flat"]
    if op == "grad":
        dx, dw_weak = owq.linear_integer_backward(s["layers"][0], s["xs"][0], s["dy"], workspace=s["workspace"])
        return {"dx": dx, "dw_weak": dw_weak}
    if op == "batched":
        return owq.linear_integer_batched(s["layers"], s["xs"], workspace=s["workspace"])
    return owq.linear_integer(s["layers"][0], s["xs"][0], workspace=s["workspace"])


# ------------------------------------------------------------------ in 64 bits


def _exact_linear(layer, x):
    M, K = x.shape
    keep = torch.ones(K, dtype=torch.bool, device=DEV)
    keep[layer["weak_idx"].long()] = False
    cols = torch.nonzero(keep).flatten()
    y = x[:, ~keep].double() @ layer["w_weak"].double().t()
    if cols.numel() == 0:
        return y
    v = x.index_select(1, cols).double()
    top = v.abs().max(dim=1).values
    # the scale and the factor are 32-bit numbers, and so is each product before it is rounded
    factor = (127.0 / top).float().double()
    scale = (top / 127.0).float().double()
    q = (v * factor[:, None]).float().double().round()
    q = torch.where(top[:, None] > 0, q, torch.zeros_like(q))
    w = layer["codes"].index_select(1, cols).double()
    return y + torch.matmul(q, w.t()) * torch.outer(scale, layer["scales"].double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        flat, views = _arena(_shapes(case), torch.float64)
        a, b, c = COEFFICIENTS
        for u, v, scale in zip(s["updates"], views, s["scales"]):
            t = u.shape[0] > u.shape[1]
            X = (u.t() if t else u).double().contiguous()
            X /= torch.linalg.vector_norm(X) + EPS
            eye = torch.eye(X.shape[0], dtype=torch.float64, device=DEV)
            for _ in range(STEPS):
                A = torch.matmul(X, X.t())
                X = torch.matmul(a * eye + b * A + c * torch.matmul(A, A), X)
            v += scale * (X.t() if t else X)
        return flat
    if case["op"] == "grad":
        layer, dy = s["layers"][0], s["dy"].double()
        W = layer["codes"].double() * layer["scales"].double()[:, None]
        W[:, layer["weak_idx"].long()] = layer["w_weak"].double()
        xw = s["xs"][0].index_select(1, layer["weak_idx"].long()).double()
        return {"dx": torch.matmul(dy, W), "dw_weak": torch.matmul(dy.t(), xw)}
    ys = [_exact_linear(L, x) for L, x in zip(s["layers"], s["xs"])]
    return ys if case["op"] == "batched" else ys[0]
