"""The choice of the next beams in float64 with exact sums (test infrastructure only)."""
import math

import numpy as np


def select(z, scores, n):
    """z [B, beams, V] float64, scores [B, beams]: (score, parent, token), each [B, n]."""
    B, beams, V = z.shape
    out = np.full((B, n), -np.inf), np.full((B, n), -1), np.full((B, n), -1)
    for b in range(B):
        best = []
        undefined = False
        for k in range(beams):
            s, row = float(scores[b, k]), z[b, k]
            if s == -math.inf:
                continue
            if not s < math.inf or np.isnan(row).any() or row.max() == np.inf:
                undefined = True
                continue
            M = row.max()
            if M == -np.inf:
                continue
            log_sum = math.log(math.fsum(np.exp(row - M)))
            order = np.argsort(-row, kind="stable")[:n]
            best += [(-math.fsum((s, row[v], -M, -log_sum)), k, int(v)) for v in order
                     if row[v] > -np.inf]
        if undefined:
            out[0][b] = np.nan
            continue
        for i, (s, k, v) in enumerate(sorted(best)[:n]):
            out[0][b, i], out[1][b, i], out[2][b, i] = -s, k, v
    return out
