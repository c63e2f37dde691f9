"""The integer form and the orthogonalised update in 64 bits, and the tolerances that
follow from the roundings the kernels are allowed."""
import torch

DEV = "cuda:0"
HALF = 2.0 ** -11      # half a step of fp16, relative
TINY = 2.0 ** -25      # and of its subnormals, absolute
F32 = 2.0 ** -23       # one fp32 operation whose rounding may truncate


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def weak_of(g, K, k):
    return torch.sort(torch.randperm(K, generator=g, device=DEV)[:k]).values.to(torch.int32)


def weights(g, N, K):
    return (torch.randn(N, K, generator=g, device=DEV) * 0.02).half()


def tokens(g, M, K, idx):
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, idx.long()] *= 20.0
    return x.half()


def rows_quantised(V, idx):
    """(codes fp64 [R][K], scale fp64 [R]) of the definition, each fp32 step rounded as such."""
    v = V.float().clone()
    v[:, idx.long()] = 0.0
    top = v.abs().amax(1, keepdim=True)
    full = torch.full_like(top, 127.0)   # (a division by a number, or of one, is not one division in torch)
    factor = torch.where(top > 0, full / top, torch.zeros_like(top))
    codes = torch.round(v * factor)
    return codes.double(), (top / full).double().flatten()


def product(layer, x):
    """(y, sum of the terms' magnitudes) of linear_integer in 64 bits."""
    idx = layer["weak_idx"].long()
    q, sm = rows_quantised(x, layer["weak_idx"])
    c, sn = layer["codes"].double(), layer["scales"].double()
    c = c.clone()
    c[:, idx] = 0.0
    xw, ww = x.double()[:, idx], layer["w_weak"].double()
    y = (q @ c.t()) * torch.outer(sm, sn) + xw @ ww.t()
    mag = (q.abs() @ c.abs().t()) * torch.outer(sm, sn) + xw.abs() @ ww.abs().t()
    return y, mag


def product_tolerance(y, mag, k):
    # the integer sum is exact; its conversion, two scalings, the sum over at most 64 lanes
    # and k weak terms are fp32; the result is rounded to fp16 once
    return HALF * (1 + HALF) * y.abs() + TINY + (16 + k) * F32 * mag


def check_product(layer, x, got):
    y, mag = product(layer, x)
    err = (got.double() - y).abs()
    tol = product_tolerance(y, mag, layer["weak_idx"].numel())
    assert got.shape == y.shape and bool((err <= tol).all()), \
        f"{int((err > tol).sum())} of {err.numel()} outputs off, worst {float((err / tol).max()):.3g} of the tolerance"


def dequantised(layer):
    W = layer["codes"].double() * layer["scales"].double()[:, None]
    W[:, layer["weak_idx"].long()] = layer["w_weak"].double()
    return W


def check_backward(layer, x, dy, dx, dw):
    W, idx = dequantised(layer), layer["weak_idx"].long()
    N, K = W.shape
    d = dy.double()
    if dx is not None:
        want, mag = d @ W, d.abs() @ W.abs()
        # every scaled gradient to fp16 (11 bits, or 2^-39 of the token's largest), N fp32
        # additions, one rounding of the result
        top = (d.abs() * layer["scales"].double()[None, :]).amax(1, keepdim=True)
        tol = (HALF + N * F32) * mag + HALF * (1 + HALF) * want.abs() + TINY + N * 2.0 ** -39 * 127 * top
        err = (dx.double() - want).abs()
        assert bool((err <= tol).all()), f"dx: worst {float((err / tol).max()):.3g} of the tolerance"
        # roundings that are independent of one another: the root mean square of each is
        # HALF / sqrt(3) of its value, two of them per output
        rms = float((err ** 2).mean().sqrt() / (want ** 2).mean().sqrt().clamp(min=1e-300))
        assert rms <= 2 * HALF or bool((want.abs() < 2.0 ** -14).any()), f"dx: relative rms error {rms:.3g}"
    if dw is not None:
        xw = x.double()[:, idx]
        want, mag = d.t() @ xw, d.abs().t() @ xw.abs()
        tol = dy.shape[0] * F32 * mag + 1e-45
        err = (dw.double() - want).abs()
        assert bool((err <= tol).all()), f"dw: worst {float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"


def newton_schulz(G, steps, coefficients, eps, scale):
    a, b, c = coefficients
    t = G.shape[0] > G.shape[1]
    X = (G.t() if t else G).double().contiguous()
    X = X / (X.pow(2).sum().sqrt() + eps)
    for _ in range(steps):
        A = torch.matmul(X, X.t())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    return scale * (X.t() if t else X)


def short_factor(G, steps, coefficients, eps, scale):
    """F with out = G F (or F G) in the form for short sides up to 96: scale / (|G| + eps)
    times the steps' polynomials of the Gram matrix."""
    a, b, c = coefficients
    t = G.shape[0] > G.shape[1]
    X = (G.t() if t else G).double()
    inv = 1.0 / (X.pow(2).sum().sqrt() + eps)
    S = torch.matmul(X, X.t().contiguous()) * inv * inv
    eye = torch.eye(S.shape[0], dtype=torch.float64, device=G.device)
    F = eye
    for _ in range(steps):
        Q = a * eye + b * S + c * torch.matmul(S, S)
        F = torch.matmul(F, Q)
        S = torch.matmul(torch.matmul(S, Q), Q)
    return F * inv * scale


def check_orthogonal(G, got, steps, coefficients, eps, scale):
    want = newton_schulz(G, steps, coefficients, eps, scale)
    err = float((got.double() - want).pow(2).mean().sqrt())
    size = float(want.pow(2).mean().sqrt())
    once = 2.0 ** -24 if got.dtype == torch.float32 else HALF + TINY / max(size, 1e-300)
    s = min(G.shape)
    if s <= 96:
        # out = sum over s terms of G and F in fp32: F is rounded once (half a step,
        # 2^-24), then s products and additions, each at most half a step of the terms'
        # magnitudes: (s + 1) 2^-24 sum |G| |F|. For a matrix of low rank F is up to a^steps
        # along the directions that G lacks, and the sum cancels.
        F = short_factor(G, steps, coefficients, eps, scale).abs()
        mag = torch.matmul(F, G.double().abs()) if G.shape[0] <= G.shape[1] else torch.matmul(G.double().abs(), F)
        bound = (s + 1) * 2.0 ** -24 * float(mag.pow(2).mean().sqrt()) + once * size
    else:
        # An error of one fp32 rounding of a matrix whose largest singular value is about
        # one grows by the step's slope, at most |a| (its value at 0), in each later step.
        bound = (2.0 ** -24 * max(abs(coefficients[0]), 1.0) ** steps + once) * size
    assert err <= bound, f"relative rms error {err / size:.3g}, tolerance {bound / size:.3g}"
    top = float((got.double() - want).abs().max())
    assert top <= 64 * bound * max(1.0, float(want.abs().max()) / size), f"largest error {top:.3g}"
