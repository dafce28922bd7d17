"""float64 / integer restatement of the AdamW step and of its 8-bit moments
(test infrastructure only).  The code of an 8-bit moment is found among all 256
values that its block can hold, not by arithmetic on its bits."""
import numpy as np

BLOCK = 128
DEPTH = {"m": 14, "v": 30}


def _mix(x, key):
    low = 0xFFFFFFFF
    x = (x ^ key) & low
    x ^= x >> 16
    x = x * 0x6A09E667 & low
    x ^= x >> 15
    x = (x + key) & low
    x = x * 0xBB67AE85 & low
    return x ^ (x >> 16)


def draws(seed, tensor, n):
    """Per element: 20 bits for m, 20 for v, 16 for a bf16 parameter (Python integers)."""
    if seed is None:
        return [1 << 19] * n, [1 << 19] * n, None
    seed &= (1 << 64) - 1
    key = _mix((seed >> 32) ^ _mix(seed & 0xFFFFFFFF, 0x9E3779B9), 0x3C6EF372)
    key = _mix(key ^ tensor, 0xDAA66D2B)
    h = [_mix(i & 0xFFFFFFFF, (key + (i >> 32) * 0x9E3779B9) & 0xFFFFFFFF) for i in range(n)]
    return ([(x >> 16) << 4 | 8 for x in h], [(x & 0xFFFF) << 4 | 8 for x in h],
            [_mix(x, key ^ 0xA54FF53A) >> 16 for x in h])


def values(top, kind):
    """What the codes from 0 stand for in a block whose largest has exponent field `top`."""
    count = 127 if kind == "m" else 255
    base = max(8 * (top - DEPTH[kind]), 0)
    bits = (np.arange(1, count, dtype=np.int64) + base) << 20
    bits = np.concatenate([[0], bits[bits < 1 << 31]])
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def decode(state, n, kind):
    out = np.empty(n)
    for b in range(-(-n // BLOCK)):
        table = values(int(state[n + b]), kind)
        for i in range(b * BLOCK, min(n, (b + 1) * BLOCK)):
            c = int(state[i])
            sign = -1.0 if kind == "m" and c & 128 else 1.0
            c = c & 127 if kind == "m" else c
            out[i] = np.nan if c == (127 if kind == "m" else 255) else sign * table[c]
    return out


def encode(x, draw, kind):
    """x float32 [n] -> state uint8 [n + blocks]."""
    n = len(x)
    blocks = -(-n // BLOCK)
    state = np.zeros(n + blocks, np.uint8)
    for b in range(blocks):
        part = np.asarray(x[b * BLOCK:(b + 1) * BLOCK], np.float32)
        a = np.abs(part.astype(np.float64))
        fin = a[np.isfinite(a)]
        largest = np.float32(fin.max() if fin.size else 0.0)
        top = int(largest.view(np.uint32)) >> 23
        state[n + b] = top
        table = values(top, kind)
        for i in range(len(part)):
            sign = 128 if kind == "m" and np.signbit(part[i]) else 0
            if not np.isfinite(part[i]):
                state[b * BLOCK + i] = sign | (127 if kind == "m" else 255)
                continue
            u = draw[b * BLOCK + i] / 2.0**20
            c = int(np.searchsorted(table, a[i], side="right")) - 1  # table[c] <= a
            if c == 0:
                if kind == "m":
                    c = int(a[i] > u * table[1])
                else:
                    c = int(a[i] > 0)
            elif c + 1 < len(table):
                c += (a[i] - table[c]) / (table[c + 1] - table[c]) + u >= 1.0
            state[b * BLOCK + i] = sign | c
    return state


def moments(m, v, g, factor, beta1, beta2):
    """fp32 m and v by products and sums rounded once each."""
    f = np.float32
    b1, c1, b2, c2 = f(beta1), f(1 - beta1), f(beta2), f(1 - beta2)
    with np.errstate(all="ignore"):
        g = np.asarray(g, f) * f(factor)
        return np.asarray(m, f) * b1 + g * c1, np.asarray(v, f) * b2 + (g * g) * c2


def parameter(p, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """float64 from the moments as they are before they are coded."""
    p, m, v = (np.asarray(x, np.float64) for x in (p, m, v))
    with np.errstate(all="ignore"):
        update = (m / (1 - beta1**step)) / (np.sqrt(v / (1 - beta2**step)) + eps)
        return p * (1 - lr * weight_decay) - lr * update
