"""The choice of the next beams where the rows of a search lie at different offsets, which a
softmax does not depend on, and scores differ by little.

Two continuations' scores, each a sum z - M + (s - ln S) of pairs of floats, are off by at most 2^-46
(|score| + 2 |s| + 28) for the roundings and 2^-40 for ln S (beams.cu), together below 2^-38 for
the scores up to 30 of these tests: scores 2^-37 apart have to come out in order."""
import numpy as np
import pytest
import torch

from test_gpu_beams import BF16, F32, _check

pytestmark = pytest.mark.gpu


def _scores(beams, seed, sign):
    """Some 2^-14 each, 2^-37 apart, in any order."""
    order = np.random.default_rng(seed).permutation(beams)
    s = sign * (np.float32(2.0**-14) + order.astype(np.float32) * np.float32(2.0**-37))
    assert len(set(s.tolist())) == beams
    return torch.tensor(s, dtype=F32, device="cuda").view(1, beams)


@pytest.mark.parametrize("offset", [1e3, 1e4, 1e5, 1e6, -1e6])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_rows_at_different_offsets(cuda_lib, offset, sign, n):
    """The same row, its columns in another order, at multiples of an offset."""
    V, beams = 6000, 6
    gen = torch.Generator(device="cuda").manual_seed(int(abs(offset)))
    base = torch.randint(-80, 40, (V,), generator=gen, device="cuda").float() / 8
    z = torch.stack([base[torch.randperm(V, generator=gen, device="cuda")] + k * offset / 4
                     for k in range(beams)])
    for k in range(beams):  # no logit was rounded
        assert torch.equal((z[k].double() - k * offset / 4).sort()[0], base.double().sort()[0])
    for seed in range(3):
        _check(cuda_lib, z, _scores(beams, seed, sign), n)


@pytest.mark.parametrize("sign", [1, -1])
def test_bf16_rows_at_different_offsets(cuda_lib, sign):
    V, beams = 5000, 4
    gen = torch.Generator(device="cuda").manual_seed(2)
    base = -2.0 * torch.randint(0, 100, (V,), generator=gen, device="cuda")
    z = torch.stack([base[torch.randperm(V, generator=gen, device="cuda")] + off
                     for off in (0, 512, -56, 200)]).to(BF16)
    assert torch.equal(z.double().sort()[0], torch.stack([base + o for o in (0, 512, -56, 200)]).double().sort()[0])
    for seed in range(3):
        _check(cuda_lib, z, _scores(beams, seed, sign), 16)


def test_scores_of_a_long_search(cuda_lib):
    """Scores of some hundreds, a step of fp32 apart, and rows at an offset."""
    V, beams = 4000, 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randint(-80, 40, (V,), generator=gen, device="cuda").float() / 8
    z = torch.stack([base[torch.randperm(V, generator=gen, device="cuda")] + k * 250000 for k in range(beams)])
    s = np.float32(-700) + np.float32(2.0**-14) * np.array([3, 0, 4, 1, 2], np.float32)
    _check(cuda_lib, z, torch.tensor(s, device="cuda").view(1, beams), 24)
