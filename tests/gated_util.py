"""The gated feed-forward block in 64 bits, for the tests."""
import numpy as np
from scipy.special import erfc

SQRT2 = np.sqrt(2.0)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def act(name, v):
    """(value, slope) of the activation."""
    if name == "silu":
        p = sigmoid(v)
        return v * p, p * (1.0 + v * (1.0 - p))
    if name == "gelu":
        p = 0.5 * erfc(-v / SQRT2)
        return v * p, p + v * np.exp(-0.5 * v * v) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        c = 2.0 * np.sqrt(2.0 / np.pi)
        p = sigmoid(c * (v + 0.044715 * v ** 3))
        return v * p, p + v * p * (1.0 - p) * c * (1.0 + 3 * 0.044715 * v * v)
    return np.maximum(v, 0.0), (v > 0).astype(np.float64)


def weights(layer):
    """fp64 [N][K] weights of a packed layer dict (device tensors), weak columns in place."""
    import oracle
    q = layer["qcodes"].cpu().numpy().view(np.uint32)
    N, G, _ = q.shape
    codes = oracle.unpack_codes(q, G * 32).astype(np.float64)
    W = (codes - layer["zeros"].cpu().numpy().astype(np.float64)[:, None])
    W = W * layer["scales"].cpu().numpy().astype(np.float64)[:, None]
    idx = layer["weak_idx"].cpu().numpy()
    W[:, idx] += layer["w_weak"].cpu().numpy().astype(np.float64)
    return W
