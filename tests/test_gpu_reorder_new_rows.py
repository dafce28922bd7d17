"""Reordering into results that the call makes itself: a row without a parent, as beam_select
leaves them where no continuation is left, is zeros, whatever the memory held."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _poison(x, rows):
    """Leaves NaN (or 0x55) in what the allocator hands out next for such a result."""
    y = torch.empty((rows, *x.shape[1:]), dtype=x.dtype, device="cuda")
    y.view(-1).view(torch.uint8).fill_(0x7F) if y.dtype != torch.bool else y.fill_(True)
    del y


def _want(x, parents):
    B, n = parents.shape
    beams = x.shape[0] // B
    ok = (parents >= 0) & (parents < beams)
    rows = parents.clamp(0, beams - 1) + torch.arange(B, device="cuda")[:, None] * beams
    out = x[rows.view(-1)]
    out[~ok.view(-1)] = 0
    return out


@pytest.mark.parametrize("beams,new", [(1, 1), (3, 3), (4, 9), (8, 5), (17, 40), (64, 128)])
@pytest.mark.parametrize("dtype", [torch.uint8, BF16, F32, torch.float64, torch.int64, torch.bool])
def test_rows_without_a_parent_are_zeros(cuda_lib, beams, new, dtype):
    B = 3
    g = torch.Generator(device="cuda").manual_seed(beams + new)
    parents = torch.randint(-1, beams, (B, new), generator=g, device="cuda")
    parents[1] = -1
    parents[0, 0] = 0
    shapes = [(), (1,), (3,), (257, 5), (4, 33, 16)]
    cache = torch.randint(0, 2, (B * beams, 4, 50, 16), generator=g, device="cuda").to(dtype)
    states = [torch.randint(0, 2, (B * beams, *s), generator=g, device="cuda").to(dtype) for s in shapes]
    states += [cache[:, :, :37], cache[:, ::2, 1:38, 3:], cache[:, :, :9].transpose(1, 3)]
    err = cuda_lib.new_error_flag("cuda:0")
    for x in states:  # alone (the native marshalling), with memory that is known to be dirty
        _poison(x, B * new)
        got, = cuda_lib.beam_reorder([x], parents, dev_error=err)
        assert torch.equal(got, _want(x, parents)), x.shape
    got = cuda_lib.beam_reorder(states, parents, dev_error=err)
    assert all(torch.equal(a, _want(x, parents)) for a, x in zip(got, states))
    assert err.item() == 0


def test_parents_out_of_range(cuda_lib):
    x = torch.randn(6, 1000, device="cuda")
    for bad in (3, -2, 1 << 40, -(1 << 40)):
        parents = torch.tensor([[2, bad, 0], [1, 1, -1]], device="cuda")
        err = cuda_lib.new_error_flag("cuda:0")
        _poison(x, 6)
        got, = cuda_lib.beam_reorder([x], parents, dev_error=err)
        assert err.item() == cuda_lib.DEV_BAD_PARAM
        assert torch.equal(got, _want(x, parents))
        kept = torch.full_like(x, 7.0)  # given results keep what they held
        cuda_lib.beam_reorder([x], parents, out=[kept])
        assert bool((kept[[1, 5]] == 7).all()) and torch.equal(kept[[0, 2, 3, 4]], got[[0, 2, 3, 4]])


def test_a_search_that_ran_out(cuda_lib):
    """What beam_select returns where no continuation is left, straight into the reordering."""
    z = torch.full((4, 100), -math.inf, device="cuda")
    z[1, 5], z[1, 7] = 1.0, 0.5
    scores, parent, token = cuda_lib.beam_select(z, torch.zeros(2, 2, device="cuda"), 3)
    assert parent.tolist() == [[1, 1, -1], [-1, -1, -1]]
    x = torch.randn(4, 2, 300, device="cuda")
    _poison(x, 6)
    got, = cuda_lib.beam_reorder([x], parent)
    assert torch.equal(got, torch.stack([x[1], x[1]] + [torch.zeros_like(x[0])] * 4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again, = cuda_lib.beam_reorder([x], parent)
    again.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, got)


def test_states_without_rows(cuda_lib):
    """No parent lies among no beams: refused, as nothing could be returned."""
    for out in (None, [torch.ones(2, 5, device="cuda")]):
        with pytest.raises(ValueError):
            cuda_lib.beam_reorder([torch.zeros(0, 5, device="cuda")],
                                  torch.zeros(1, 2, dtype=torch.int64, device="cuda"), out=out)
