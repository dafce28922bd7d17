"""e4m3 matrices with a scale per block, in float64 (test infrastructure only).  The nearest
code is found among all values of the type."""
import numpy as np

BLOCK = 128


def e4m3_values():
    """The finite values of codes 0..126, ascending."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m / 8 * 2.0**-6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def nearest(x):
    """x rounded to e4m3, ties to the even code; |x| <= 448."""
    table = e4m3_values()
    a = np.abs(x)
    lo = np.searchsorted(table, a, side="right") - 1
    hi = np.minimum(lo + 1, len(table) - 1)
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (lo % 2 == 1))
    return np.copysign(np.where(up, table[hi], table[lo]), x)


def quantize(x, rows):
    """(values over the scale, scales) of x float64 [T, K]."""
    T, K = x.shape
    q = np.zeros((T, K))
    s = np.ones((-(-T // rows), -(-K // BLOCK)))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = slice(i * rows, (i + 1) * rows), slice(j * BLOCK, (j + 1) * BLOCK)
            block = x[at]
            if not np.isfinite(block).all():
                s[i, j] = np.nan
                continue
            top = np.abs(block).max()
            if top > 0:
                e = -126
                while 448.0 * 2.0**e < top:
                    e += 1
                s[i, j] = 2.0**e
            q[at] = nearest(block / s[i, j])
    return q, s
