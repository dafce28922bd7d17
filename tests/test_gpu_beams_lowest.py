"""The choice of the next beams with masks and scores of the type's lowest value, whose sums lie
below fp32's range: a continuation that does counts as masked, and none of them
comes before one that does not."""
import math

import numpy as np
import pytest
import torch

from oracle import beams as obeams
from test_gpu_beams import BF16, F32

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(F32).min


def _run(lib, z, scores, n):
    err = lib.new_error_flag("cuda:0")
    got = [x.cpu().numpy() for x in lib.beam_select(z, scores, n, dev_error=err)]
    assert err.item() == 0
    B, beams = scores.shape
    want = obeams.select(z.double().cpu().numpy().reshape(B, beams, -1), scores.cpu().numpy(), n)
    gone = want[0] < LOWEST * (1 + 2.0**-25)  # what rounds to -inf in fp32
    for x, none in zip(want, (-math.inf, -1, -1)):
        x[gone] = none
    return got, want


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [4, 9, 40])
@pytest.mark.parametrize("beams", [1, 3])
def test_beams_and_columns_of_the_lowest_value(cuda_lib, dtype, n, beams):
    """All beams but the first at the lowest score; in all rows seven columns that are not
    masked."""
    V = 3000
    gen = torch.Generator(device="cuda").manual_seed(n)
    z = torch.full((2 * beams, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    z[:, 100:2200:300] = (3 * torch.randn(2 * beams, 7, generator=gen, device="cuda")).to(dtype)
    s = torch.full((2, beams), LOWEST, device="cuda")
    (score, parent, token), (ws, wp, wt) = _run(cuda_lib, z, s, n)  # no beam is left
    assert not np.isnan(score).any()
    open_ = min(n, 7 * beams)
    for b in range(2):
        # the scores are alike to the last bit of fp32, so their order is open; the masked
        # columns' are below its range (bf16: finfo.min of bf16 and of fp32 together)
        at = {(k, v) for k, v in zip(parent[b, :open_].tolist(), token[b, :open_].tolist())}
        assert len(at) == open_ and at <= {(k, v) for k in range(beams) for v in range(100, 2200, 300)}
        assert (score[b, :open_] == np.float32(LOWEST)).all()
        assert (score[b, open_:] == -math.inf).all()
        assert (parent[b, open_:] == -1).all() and (token[b, open_:] == -1).all()
    s[:, 0] = -2.0
    (score, parent, token), (ws, wp, wt) = _run(cuda_lib, z, s, n)
    k = min(n, 7)
    assert np.array_equal(parent[:, :k], wp[:, :k]) and np.array_equal(token[:, :k], wt[:, :k])
    assert (np.abs(score[:, :k] - ws[:, :k]) <= 6e-6 + 2.0**-24 * np.abs(ws[:, :k])).all()
    assert not np.isnan(score).any() and (score[:, k:] < -3e38).all()


def test_rows_far_from_their_masks(cuda_lib):
    """Maxima so large that the masked columns' distance is below fp32's range, and rows so
    low that score - M alone is above it."""
    V = 2500
    z = torch.full((4, V), LOWEST, device="cuda")
    z[0, 7], z[0, 1200] = 1e33, 0.0
    z[1, 3], z[1, 2400] = 3e38, 2.9e38
    z[2] = -1e38
    z[2, 5:] = -math.inf
    z[3, 11] = 1e32
    s = torch.tensor([[-1.0, -2.0, 3e38, -math.inf]], device="cuda")
    (score, parent, token), (ws, wp, wt) = _run(cuda_lib, z, s, 40)
    assert np.array_equal(parent, wp), (parent, wp)
    assert np.array_equal(token, wt), (token, wt)
    fin = np.isfinite(ws)
    assert fin.sum() == 9 and np.array_equal(score[~fin], ws[~fin])
    assert (np.abs(score[fin].astype(np.float64) - ws[fin]) <= 6e-6 + 2.0**-24 * np.abs(ws[fin])).all()
