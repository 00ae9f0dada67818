"""The fp32 scans' split of a factor into two tf32 numbers, emulated: both are
numbers that the instruction takes, and what they leave out is within the stated
bounds."""

import numpy as np

MASK = np.uint32(0xFFFFE000)


def split(x):
    hi = ((x.view(np.uint32) + np.uint32(0x1000)) & MASK).view(np.float32)
    lo = ((x - hi).view(np.uint32) & MASK).view(np.float32)
    return hi, lo


def test_split():
    n = np.arange(1 << 23, dtype=np.uint32)
    for exponent in (127, 100, 254):  # every number of a binade; the largest one's last numbers round up to infinity
        x = (n | np.uint32(exponent << 23)).view(np.float32)
        if exponent == 254:
            x = x[x < np.float32(3.39e38)]
        for y in (x, -x):
            hi, lo = split(y)
            assert not (hi.view(np.uint32) & ~MASK).any() and not (lo.view(np.uint32) & ~MASK).any()
            assert (np.abs(lo) <= np.abs(y) * np.float32(2.0 ** -11)).all()
            # (exact: differences of neighbours in fp32)
            left = np.abs((y - hi) - lo).astype(np.float64)
            assert (left <= 2.0 ** -23 * np.abs(y.astype(np.float64))).all() and left.max() > 0
