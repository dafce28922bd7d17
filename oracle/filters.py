"""Float64 oracle for tempered, truncated distributions and gradient clipping.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Row z, temperature t, M = max z, x = (z - M)/t, e = exp(x).  Tokens ordered by
(logit descending, index ascending), -inf never kept; top-k keeps the first
k, top-p the shortest prefix whose mass reaches p times what top-k left,
min-p the tokens with x >= ln(min_p); the kept set is the shortest of them.
Settings are taken at their float32 values, which is what the kernels get.
"""
from __future__ import annotations

import math

import numpy as np


def to_double(z):
    """A float32 array, or bf16 bit patterns (uint16), as float64."""
    z = np.asarray(z)
    if z.dtype == np.uint16:
        z = (z.astype(np.uint32) << 16).view(np.float32)
    return z.astype(np.float64)


def _f32(x):
    return float(np.float32(x))


def kept_set(z, t=1.0, k=0, p=1.0, m=0.0):
    """(kept mask, cut logit, cut index, x, e) of one row of float64 logits."""
    t, p, m = _f32(t), _f32(p), _f32(m)
    z = z + 0.0
    V = len(z)
    finite = np.isfinite(z)
    M = z[finite].max()
    with np.errstate(over="ignore"):
        x = (z - M) / t
    e = np.exp(x)
    free = not (0 < k < V) and p >= 1.0 and m <= 0.0
    order = np.lexsort((np.arange(V), -z))
    n = int(finite.sum())
    if 0 < k < n:
        n = k
    j = n
    if p < 1.0:
        total = math.fsum(e[order[:n]])
        acc = np.cumsum(e[order[:n]])
        j = min(n, int(np.searchsorted(acc, p * total, side="left")) + 1)
    if m > 0.0:
        j = min(j, int((x >= math.log(m)).sum()))
    kept = np.zeros(V, bool)
    kept[order[:j]] = True
    if free:
        return kept, -math.inf, V - 1, x, e
    last = order[j - 1]
    return kept, z[last], int(last), x, e


def sample(z, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob, distance) of one row; `distance` is how far the target
    u S is from the nearest border of the cumulative mass, relative to S."""
    u = _f32(u)
    if t == 0:
        return int(np.argmax(z)), 0.0, math.inf
    kept, _, _, x, e = kept_set(z, t, k, p, m)
    acc = np.cumsum(np.where(kept, e, 0.0))
    S = acc[-1]
    v = int(np.searchsorted(acc, u * S, side="right"))
    return v, x[v] - math.log(S), float(np.min(np.abs(acc - u * S)) / S)


def forward(z, y, t=1.0, k=0, p=1.0, m=0.0, ignore_index=-100):
    """dict of one row's logprob, entropy, M, lnS, cut logit and index."""
    kept, tau, index, x, e = kept_set(z, t, k, p, m)
    S = math.fsum(e[kept])
    lnS = math.log(S) if S >= 2 else math.log1p(math.fsum(e[kept][e[kept] < 1.0])
                                                + float((e[kept] == 1.0).sum() - 1))
    H = lnS - math.fsum(e[kept & (e > 0)] * x[kept & (e > 0)]) / S
    if y == ignore_index:
        lp = 0.0
    else:
        lp = x[y] - lnS if kept[y] and np.isfinite(z[y]) else -math.inf
    return {"logprob": lp, "entropy": H, "M": float(z[np.isfinite(z)].max()), "lnS": lnS,
            "cut_logit": tau, "cut_index": index}


def backward(z, y, w, t=1.0, k=0, p=1.0, m=0.0, ignore_index=-100):
    """dlogits of one row."""
    kept, _, _, x, e = kept_set(z, t, k, p, m)
    g = np.zeros(len(z))
    if y == ignore_index or w == 0 or not kept[y]:
        return g
    g[kept] = -e[kept] / math.fsum(e[kept])
    g[y] += 1.0
    return g * (float(w) / _f32(t))


def grad_norm(arrays):
    """L2 norm over a list of arrays, without overflow or underflow."""
    arrays = [to_double(a).ravel() for a in arrays]
    big = max((float(np.abs(a).max()) for a in arrays if a.size), default=0.0)
    if big == 0.0 or not math.isfinite(big):
        return big
    return big * math.sqrt(math.fsum(float(np.dot(a / big, a / big)) for a in arrays if a.size))
