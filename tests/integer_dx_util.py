"""How close dx of the integer form's backward has to be: the formula in 64 bits, on any
device, with bounds far below one row's part of a sum."""
import torch

HALF = 2.0 ** -11      # half a step of fp16, relative
TINY = 2.0 ** -25      # and of its subnormals, absolute
# A scaled gradient is one fp32 product (2^-24) and a pair of fp16 values, each half a step
# of what is left: 2^-11 of 2^-11.
PAIR = 2.0 ** -22 + 2.0 ** -24


def exact_dx(codes, scales, w_weak, weak_idx, dy):
    """(dx, root of the sum of the squared terms) in 64 bits."""
    W = codes.double() * scales.double()[:, None]
    W[:, weak_idx.long()] = w_weak.double()
    d = dy.double()
    return d @ W, ((d * d) @ (W * W)).sqrt()


def faults(codes, scales, w_weak, weak_idx, dy, dx):
    """What is wrong with dx, as a list of texts; empty for a good one.

    Each: the terms' signs are independent of their sizes, so partial sums stay within some
    four times the root of the squared terms (rss); N / 8 additions per output that may truncate
    (2^-23 of the partial sum each), and the result is rounded once. The smallest scaled
    gradients are held to 2^-39 of the token's largest.
    All: a value that is off by e before it is rounded rounds to another fp16 value with
    probability |e| / step, so the mean distance from the rounded 64-bit value is the mean of
    |e|: the pairs' error and sqrt(N) additions' worth of it, twice that as the limit."""
    N = codes.shape[0]
    want, rss = exact_dx(codes, scales, w_weak, weak_idx, dy)
    top = (dy.double().abs() * scales.double()[None, :]).amax(1, keepdim=True)
    floor = N * 2.0 ** -39 * 127 * top
    err = (dx.double() - want).abs()
    tol = HALF * (1 + HALF) * want.abs() + TINY + (2 * PAIR + N / 8 * 2.0 ** -23) * 4 * rss + floor
    out = []
    if not bool((err <= tol).all()):
        out.append(f"{int((~(err <= tol)).sum())} of {err.numel()} values off, worst "
                   f"{float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance")
    off = float((dx.double() - want.half().double()).abs().mean())
    # (one value lies a whole step off by chance: a step of the largest is allowed on top)
    limit = float((2 * (PAIR + N ** 0.5 * 2.0 ** -23) * rss + floor).mean()) \
        + float((2 * HALF * want.abs() + 2 * TINY).max()) / want.numel()
    if not off <= limit:
        out.append(f"mean distance from the rounded value {off:.3g}, limit {limit:.3g}")
    return out
