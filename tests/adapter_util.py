"""Cases of the adapted linear whose tolerance is far below the adapters' part, and
that tolerance, for the tests.

  y = s + alpha sum_c B[c] t[c],  s = sum_j W[j] x[j],  t[c] = sum_j A[c][j] x[j]

Tolerance of an output:
  * s is an fp32 sum of exact products with a chain of at most K / 4 + 64 roundings
    (as in the gated block's tests): (K / 4 + 64) 2^-24 S, S its sum of absolute terms.
  * t[c] is an fp32 sum of exact products. Sixteen waves share the 32-column steps and
    have two accumulators each, so a chain is at most 32 ceil(steps / 32) roundings of
    products, one more for the two accumulators and 16 for the waves: dt = that times
    2^-24 sum_j |A[c][j] x[j]|. Where all sums of absolute terms stay below 2^24 units
    of integers, every partial sum is exact and dt = 0.
  * t goes on as two fp16 values after scaling the row's largest into [2^14, 2^15):
    the first leaves at most 2^-11 |t| (half a step), the second 2^-11 of that or half
    its smallest subnormal, 2^-25 against 2^14: 2^-22 |t[c]| + 2^-39 max |t|.
  * the second sum has at most 2 rank products, each with one rounding, their factor
    alpha (2), the partial sums of 16 ranks (rank / 16 + 2), s (1) and, where lanes
    share the sum, their reduction (6): (2 rank + rank / 16 + 16) 2^-24 of alpha
    sum_c |B[c]| (|t[c]| + dt), and 8 more roundings of s's absolute terms.
  * the result is rounded to fp16: 2^-11 |y|, or half its smallest subnormal 2^-25."""
import math

import numpy as np

SPLIT_BITS = 22


def zero_layer(N, K, k):
    """A packed layer (numpy) of zero weights: y is the adapters' part alone."""
    return {"qcodes": np.zeros((N, K // 32, 3), np.uint32), "scales": np.full(N, 1.0, np.float16).view(np.uint16),
            "zeros": np.zeros(N, np.uint8), "weak_idx": np.arange(k, dtype=np.int32) * (K // max(k, 1)),
            "w_weak": np.zeros((N, k), np.uint16)}


def device_layer(layer):
    from parity_util import dev
    return {"qcodes": dev(layer["qcodes"].view(np.int32)), "scales": dev(layer["scales"].view(np.float16)),
            "zeros": dev(layer["zeros"]), "weak_idx": dev(layer["weak_idx"]),
            "w_weak": dev(layer["w_weak"].reshape(len(layer["zeros"]), -1).view(np.float16))}


def dense(layer):
    """fp64 [N][K] weights of a packed layer."""
    import oracle
    N, G, _ = layer["qcodes"].shape
    W = oracle.unpack_codes(layer["qcodes"], 32 * G).astype(np.float64) - layer["zeros"].astype(np.float64)[:, None]
    W = W * layer["scales"].view(np.float16).astype(np.float64)[:, None]
    W[:, layer["weak_idx"]] += layer["w_weak"].reshape(N, -1).view(np.float16).astype(np.float64)
    return W


def requests(name, M, count, rng):
    return {"mixed": rng.integers(-1, count, M), "one": np.full(M, count - 1),
            "runs": np.arange(M) * (count + 1) // M - 1}[name].astype(np.int32)


def cancelling(N, K, k, M, rank, count, which, seed):
    """A zero layer, and adapters whose products nearly cancel: every row of B is
    orthogonal to its adapter's t up to B's rounding, and t are integers of 15 to 20
    bits, so that bits of t below fp16's eleven decide the output. A token's x is its
    adapter's one vector times a power of two and a sign."""
    rng = np.random.default_rng(seed)
    top = int(math.sqrt(2.0 ** 24 / K))  # sums of absolute products stay below 2^24 units
    top = min(top, 1024)
    v = rng.integers(-top, top + 1, (count, K)).astype(np.float64)
    A = rng.integers(-top, top + 1, (count, rank, K)).astype(np.float64)
    t = np.einsum("rck,rk->rc", A, v)
    B = 0.25 * rng.standard_normal((count, N, rank))
    if rank > 1:
        B -= (B @ t[:, :, None]) / np.sum(t * t, axis=1)[:, None, None] * t[:, None, :]
    else:
        B *= 2.0 ** -8
    alpha = (0.5 + 1.5 * rng.random(count)).astype(np.float32)
    x = rng.integers(-top, top + 1, (M, K)).astype(np.float64)
    for m, r in enumerate(which):
        if 0 <= r < count:
            x[m] = v[r] * 2.0 ** rng.integers(-3, 1) * rng.choice([-1.0, 1.0])
    # rows of A of one adapter in one power of two: far below fp16's range of products, or above
    A *= 2.0 ** rng.choice([-14, -7, 0], count)[:, None, None]
    B *= 2.0 ** -4
    return zero_layer(N, K, k), x.astype(np.float16), A.astype(np.float16), B.astype(np.float16), alpha


def beside(N, K, k, M, rank, count, which, seed):
    """A random layer, its weights and B so large that the adapters' part is a good share of the output."""
    import oracle
    rng = np.random.default_rng(seed)
    W = ((0.02 if K <= 8192 else 0.001) * rng.standard_normal((N, K))).astype(np.float16)
    idx = np.sort(rng.choice(K, k, replace=False)).astype(np.int32)
    A = (rng.standard_normal((count, rank, K)) / np.sqrt(K)).astype(np.float16)
    B = rng.standard_normal((count, N, rank)).astype(np.float16)
    alpha = (0.5 + 1.5 * rng.random(count)).astype(np.float32)
    x = rng.standard_normal((M, K)).astype(np.float16)
    return oracle.pack(W, idx), x, A, B, alpha


def reference(layer, x, A, B, alpha, which, exact_t, t_bits=None, share=1.0):
    """(y, tolerance, the adapters' part of y), in 64 bits. t_bits: t rounded to so many bits; share: of the adapters'
    part that is added (mistakes, for the test of the tolerance)."""
    M, K = x.shape
    rank = A.shape[1]
    W, x64 = dense(layer), x.astype(np.float64)
    y, S = x64 @ W.T, np.abs(x64) @ np.abs(W).T
    tol = (K / 4 + 64 + 8) * 2.0 ** -24 * S
    part = np.zeros_like(y)
    steps = K // 32
    chain = 0.0 if exact_t else 32 * math.ceil(steps / 32) + 17
    for r in set(which.tolist()):
        if not 0 <= r < len(alpha):
            continue
        m = which == r
        A64, B64, al = A[r].astype(np.float64), B[r].astype(np.float64), abs(float(alpha[r]))
        t, ta = x64[m] @ A64.T, np.abs(x64[m]) @ np.abs(A64).T
        dt = chain * 2.0 ** -24 * ta
        if t_bits:
            f, e = np.frexp(t)
            t = np.ldexp(np.rint(f * 2.0 ** t_bits) / 2.0 ** t_bits, e)
        part[m] = share * float(alpha[r]) * (t @ B64.T)
        kept = 2.0 ** -SPLIT_BITS * np.abs(t) + 2.0 ** -39 * np.max(np.abs(t), axis=1, keepdims=True)
        tol[m] += al * ((dt + kept) @ np.abs(B64).T)
        tol[m] += (2 * rank + rank / 16 + 16) * 2.0 ** -24 * al * ((np.abs(t) + dt) @ np.abs(B64).T)
    y = y + part
    return y, tol + 2.0 ** -11 * (np.abs(y) + tol) + 2.0 ** -25, part


CASES = [
    # N, K, k, M, rank, count
    (33, 32, 0, 1, 1, 1),
    (130, 64, 0, 1, 16, 8),
    (67, 1024, 4, 2, 100, 3),
    (9000, 96, 3, 1, 12, 2),
    (300, 64, 0, 3, 8, 5),
    (300, 768, 6, 4, 12, 5),
    (129, 4096, 9, 8, 64, 9),
    (200, 64, 2, 16, 33, 20),
    (70, 65536, 9, 5, 3, 2),
    # above 16 tokens, every tile of the pair product
    (513, 96, 3, 17, 4, 2),
    (190, 1024, 9, 40, 12, 3),
    (64, 64, 0, 70, 256, 2),
    (257, 64, 0, 127, 16, 40),
    (333, 96, 0, 300, 7, 130),
    (4200, 64, 3, 150, 8, 3),
    (16600, 96, 3, 50, 12, 5),
    (22000, 160, 3, 200, 3, 4),
    (20000, 96, 3, 260, 8, 3),
    (40000, 64, 3, 260, 4, 3),
]
