"""The tolerance of the adapted linear's GPU tests, held against mistakes planted in
the 64-bit reference. Beside a layer a result without the adapters, or with nine tenths
of them, is outside it in every case; alone, with products that nearly cancel, so is one
whose t has fp16's eleven bits instead of 22 (up to rank 64: the roundings that a longer
sum may make hide it)."""
import numpy as np
import pytest

import adapter_util as au


def _unit(v):
    """The largest power of two that all values of v are integer multiples of."""
    f, e = np.frexp(v.astype(np.float64)[v != 0])
    i = np.rint(np.ldexp(f, 11)).astype(np.int64)
    return 2.0 ** int(np.min(np.log2(np.abs(i & -i)) + e - 11))


@pytest.mark.parametrize("name", ["mixed", "one"])
@pytest.mark.parametrize("case", au.CASES, ids=str)
def test_mistakes_are_outside(case, name):
    N, K, k, M, rank, count = case
    which = au.requests(name, M, count, np.random.default_rng(M))
    on = which >= 0
    if not on.any():
        which[0], on[0] = 0, True
    for make in (au.cancelling, au.beside):
        args = make(*case, which, seed=sum(case))
        alone = make is au.cancelling
        if alone:  # every partial sum of x A is exact in fp32, in any order
            _, x, A, _, _ = args
            for m in np.flatnonzero(on):
                a = A[which[m]].astype(np.float64)
                s = np.abs(x[m].astype(np.float64)) @ np.abs(a).T
                assert s.max() <= 2.0 ** 24 * _unit(x[m]) * _unit(a.astype(np.float16)), m
        y, tol, part = au.reference(*args, which, alone)
        assert np.isfinite(y.astype(np.float16)).all()

        def outside(**mistake):
            return (np.abs(au.reference(*args, which, alone, **mistake)[0] - y) > tol)[on]
        assert not outside(t_bits=24).any()
        assert outside(share=0.0).any()
        if not alone:
            assert outside(share=0.9).any()
            assert np.median(tol[on]) < np.median(np.abs(part[on])) / 4
        elif 1 < rank <= 64:
            assert outside(t_bits=11).any()
