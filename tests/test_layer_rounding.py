"""The quantiser's rounding of bf16 rows, replayed in numpy's fp32: 127 t / m is first rounded to 18 bits (as
p - (p - u) with p = 65 u) and then to an integer, which has to be the nearest code of the exact quotient, ties to
even, for every pair of an 8-bit t and an 8-bit m (no GPU needed)."""
import numpy as np


def _code(t, m, split):
    f = np.float32
    inv = f(f(127) / f(m))
    if not split:
        return np.rint((t.astype(np.float64) * np.float64(inv)).astype(f))
    p = t.astype(f) * f(f(65) * inv)
    # a fused multiply-add: the product of 8 and 24 bits and the difference are exact in fp64, rounded once
    q = (p.astype(np.float64) - t * np.float64(inv)).astype(f)
    return np.rint((p.astype(np.float64) - q.astype(np.float64)).astype(f))


def _wrong(split):
    wrong = 0
    T = np.arange(128, 256, dtype=np.float64)
    for M in range(128, 256):
        for shift in range(0, 12):
            t = T * 2.0 ** -shift
            t = t[t <= M]
            wrong += int((_code(t, M, split) != np.rint(t * 127 / M)).sum())
    return wrong


def test_split_rounding_finds_the_nearest_code_of_every_pair():
    assert _wrong(split=True) == 0


def test_plain_rounding_does_not():
    """Without the split some ties go astray, which is what it is for."""
    assert _wrong(split=False) > 0
