"""The choice of the next beams against float64 with exact sums.

Parents and tokens have to be equal.  A score is off by at most 6e-6 (include/pstat.h:
the fp32 sum's 2^-18, the logarithm's 2^-20) and half a step of fp32."""
import math

import numpy as np
import pytest
import torch

from oracle import beams as obeams

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _check(lib, z, scores, n, want_error=0):
    B, beams = scores.shape
    err = lib.new_error_flag("cuda:0")
    got = lib.beam_select(z, scores, n, dev_error=err)
    assert err.item() == want_error
    want = obeams.select(z.double().cpu().numpy().reshape(B, beams, -1), scores.cpu().numpy(), n)
    score, parent, token = (x.cpu().numpy() for x in got)
    assert np.array_equal(parent, want[1]), (parent, want[1])
    assert np.array_equal(token, want[2]), (token, want[2])
    assert np.array_equal(np.isnan(score), np.isnan(want[0]))
    fin = np.isfinite(want[0])
    assert np.array_equal(score[~fin & ~np.isnan(want[0])], want[0][~fin & ~np.isnan(want[0])])
    assert (np.abs(score[fin].astype(np.float64) - want[0][fin])
            <= 6e-6 + 2.0**-24 * np.abs(want[0][fin])).all()
    return got


def _rows(T, V, dtype, seed, pad=0, off=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.zeros(T * (V + pad) + off, dtype=dtype, device="cuda")
    z = store[off:].view(T, V + pad)[:, :V]
    z.copy_(spread * torch.randn(T, V, generator=g, device="cuda"))
    return z, -10 * torch.rand(T, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,beams,n,V,pad,off", [
    (1, 1, 1, 1, 0, 0), (1, 1, 4, 3, 0, 0), (2, 3, 6, 7, 1, 1), (1, 4, 8, 151936, 0, 0),
    (3, 5, 10, 4097, 0, 0), (2, 7, 33, 10007, 9, 3), (1, 64, 128, 2000, 0, 0), (2, 16, 32, 20001, 0, 1),
    (40, 2, 4, 1000, 0, 0), (1, 2, 64, 151937, 0, 0), (1, 33, 100, 30000, 8, 0)])
def test_against_oracle(cuda_lib, dtype, B, beams, n, V, pad, off):
    z, s = _rows(B * beams, V, dtype, V + n, pad, off)
    _check(cuda_lib, z, s.view(B, beams), n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 32, 33, 128])
def test_ties(cuda_lib, dtype, n):
    """Equal logits everywhere; equal beams; logits in order, so that the best lie in few
    runs and whole groups reach the list."""
    V, beams = 9000, 3
    z = torch.full((beams, V), 1.5, dtype=dtype, device="cuda")
    s = torch.tensor([[-1.0, -1.0, -1.0]], device="cuda")
    _check(cuda_lib, z, s, n)
    s[0, 0] = -1.25
    _check(cuda_lib, z, s, n)
    up = torch.arange(V, device="cuda").float().div(700).to(dtype)
    _check(cuda_lib, up.expand(beams, V), s, n)
    _check(cuda_lib, up.flip(0).expand(beams, V), s, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_order_of_equal_and_nearly_equal_beams(cuda_lib, dtype):
    """Rows with the same logits in another order have the same sum, which fp32 sums
    do not know: every continuation ties with one of each other beam.  Then scores that
    differ by one step of fp32, 2e-6, which is less than the sums' error."""
    V, beams = 20000, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    base = (2 * torch.randn(V, generator=g, device="cuda")).to(dtype)
    z = torch.stack([base[torch.randperm(V, generator=g, device="cuda")] for _ in range(beams)])
    s = torch.full((1, beams), -20.0, device="cuda")
    _check(cuda_lib, z, s, 40)
    for k in range(beams):
        s[0, k] = float(np.float32(-20) + np.float32(1.9073486e-06) * ((k * 5) % beams))
    assert len(set(s.view(-1).tolist())) == beams
    _check(cuda_lib, z, s, 40)
    # and where the nearly equal ones straddle the end of the list
    for n in range(1, 14):
        _check(cuda_lib, z, s, n)


def test_masks_dead_beams_and_undefined_rows(cuda_lib):
    V, beams = 5000, 4
    for dtype in (BF16, F32):
        z, s = _rows(3 * beams, V, dtype, 3)
        s = s.view(3, beams)
        z[0, 10:] = -math.inf      # few continuations
        z[1] = -math.inf           # none
        s[0, 2] = s[0, 3] = -math.inf
        s[1] = -math.inf           # a search that is over
        _check(cuda_lib, z, s, 24)
        z[2, 5] = math.nan         # of a dead beam: not looked at
        z[3, 7] = math.inf
        _check(cuda_lib, z, s, 24)
        for row, bad in ((8, math.nan), (9, math.inf)):
            y = z.clone()
            y[row, 4999] = bad
            _check(cuda_lib, y, s, 24, cuda_lib.DEV_EMPTY_ROW)
        for bad in (math.nan, math.inf):
            t = s.clone()
            t[2, 1] = bad
            _check(cuda_lib, z, t, 24, cuda_lib.DEV_EMPTY_ROW)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_range(cuda_lib, dtype):
    """Peaked rows, huge and tiny logits."""
    z, s = _rows(8, 3000, dtype, 5)
    z[0, 100] = 80.0
    z[1] *= 1e30
    z[2] *= 1e-30
    z[3] = torch.where(z[3] > 0, 0.0, -1e38).to(dtype)
    s[4] = -1e30
    _check(cuda_lib, z, s.view(2, 4), 16)


def test_same_bits_in_any_batch(cuda_lib):
    z, s = _rows(24, 30011, BF16, 7)
    whole = cuda_lib.beam_select(z, s.view(6, 4), 8)
    for b in range(6):
        one = cuda_lib.beam_select(z[4 * b:4 * b + 4], s[4 * b:4 * b + 4].view(1, 4), 8)
        assert all(torch.equal(x[b:b + 1], y) for x, y in zip(whole, one))


def test_graph_stream_and_outputs(cuda_lib):
    z, s = _rows(16, 50000, BF16, 9)
    s = s.view(4, 4)
    out = (torch.empty(4, 8, device="cuda"), torch.empty(4, 8, dtype=torch.int64, device="cuda"),
           torch.empty(4, 8, dtype=torch.int64, device="cuda"))
    ws = torch.empty(cuda_lib.beam_workspace_size(4, 4, 50000, BF16), dtype=torch.uint8, device="cuda")
    count = out[0]._version
    got = cuda_lib.beam_select(z, s, 8, out=out, workspace=ws)
    assert all(a is b for a, b in zip(got, out)) and out[0]._version == count + 1
    first = [x.clone() for x in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = cuda_lib.beam_select(z, s, 8)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.beam_select(z, s, 8, out=out, workspace=ws)
    z.copy_(z.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, cuda_lib.beam_select(z, s, 8)))
    assert not torch.equal(out[2], first[2])
    empty = cuda_lib.beam_select(z[:0], s[:0], 8)
    assert empty[0].shape == (0, 8)


def test_refusals(cuda_lib):
    z, s = _rows(8, 100, F32, 1)
    s = s.view(2, 4)
    for bad in (0, 129):
        with pytest.raises(ValueError):
            cuda_lib.beam_select(z, s, bad)
    for args in ((z, s.view(-1)), (z, s[:1]), (z, s.double()), (z.t(), s), (z, s.cpu()), (z.cpu(), s)):
        with pytest.raises(ValueError):
            cuda_lib.beam_select(*args, 4)
    with pytest.raises(TypeError):
        cuda_lib.beam_select(z.half(), s, 4)
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_select(torch.zeros(65, 10, device="cuda"), torch.zeros(1, 65, device="cuda"), 4)
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_select(z, s, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cuda_lib.beam_select(z, s, 4, out=(torch.empty(2, 5, device="cuda"), None, None))


# ---- reordering --------------------------------------------------------------------


def _reordered(x, parents):
    B, n = parents.shape
    beams = x.shape[0] // B
    rows = parents + torch.arange(B, device=parents.device)[:, None] * beams
    return x[rows.reshape(-1)]


TYPES = [torch.uint8, BF16, F32, torch.float64, torch.complex128, torch.bool, torch.int16]


@pytest.mark.parametrize("beams", [1, 2, 5, 8, 9, 16, 17, 32, 33, 64])
def test_reorder(cuda_lib, beams):
    B = 3
    g = torch.Generator(device="cuda").manual_seed(beams)
    parents = torch.randint(0, beams, (B, beams), generator=g, device="cuda")
    parents[1] = torch.arange(beams, device="cuda").flip(0)  # a permutation with cycles
    states = []
    for i, t in enumerate(TYPES):
        for shape in ((), (1,), (3,), (257, 5), (4, 33, 16)):
            x = torch.randint(0, 2 if t == torch.bool else 120, (B * beams, *shape), generator=g, device="cuda")
            states.append(x.to(t))
    cache = torch.randn(B * beams, 4, 50, 16, generator=g, device="cuda").to(BF16)
    keep = cache.clone()
    wide = torch.randn(B * beams, 4, 6, 10, generator=g, device="cuda")
    states += [cache[:, :, :37], cache[:, :, 37:40], cache[:, :, 41:, 3:], wide[:, ::2, :, ::2],
               wide[:, 1::2].transpose(1, 3)]
    want = [_reordered(x, parents) for x in states]
    got = cuda_lib.beam_reorder(states, parents)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(cache, keep)
    back = cuda_lib.beam_reorder(states, parents, out=states)
    assert all(a is b for a, b in zip(back, states))
    assert all(torch.equal(a, b) for a, b in zip(states, want))
    # what lies between the views stays as it was
    assert torch.equal(cache[:, :, 40], keep[:, :, 40])
    assert torch.equal(cache[:, :, 41:, :3], keep[:, :, 41:, :3])


def test_reorder_to_more_or_fewer_beams(cuda_lib):
    for beams, new in ((4, 8), (8, 3), (1, 100), (64, 128)):
        g = torch.Generator(device="cuda").manual_seed(new)
        parents = torch.randint(0, beams, (2, new), generator=g, device="cuda")
        x = torch.randn(2 * beams, 7, 5, generator=g, device="cuda")
        got, = cuda_lib.beam_reorder([x], parents)
        assert torch.equal(got, _reordered(x, parents))


def test_reorder_without_parent(cuda_lib):
    x = torch.randn(6, 1000, device="cuda")
    parents = torch.tensor([[2, -1, 0], [1, 1, -1]], device="cuda")
    err = cuda_lib.new_error_flag("cuda:0")
    want = torch.stack([x[2], x[1], x[0], x[4], x[4], x[5]])
    y = x.clone()
    cuda_lib.beam_reorder([y], parents, out=[y], dev_error=err)
    assert torch.equal(y, want) and err.item() == 0
    z = torch.full_like(x, 7.0)
    cuda_lib.beam_reorder([x], parents, out=[z], dev_error=err)
    assert bool((z[[1, 5]] == 7).all()) and torch.equal(z[[0, 2, 3, 4]], want[[0, 2, 3, 4]])
    for bad in (3, -2, 1 << 40):
        parents[0, 1] = bad
        err.zero_()
        y = x.clone()
        cuda_lib.beam_reorder([y], parents, out=[y], dev_error=err)
        assert torch.equal(y, want) and err.item() == cuda_lib.DEV_BAD_PARAM


def test_reorder_past_32_bits(cuda_lib):
    """Rows whose offsets pass 2^32 bytes."""
    x = torch.zeros(6, (1 << 30) + 24, dtype=torch.uint8, device="cuda")
    x += torch.arange(6, dtype=torch.uint8, device="cuda")[:, None]
    x[:, -1] += 10
    parents = torch.tensor([[5, 4, 2, 0, 0, 1]], device="cuda")
    cuda_lib.beam_reorder([x], parents, out=[x])
    assert x[:, 0].tolist() == [5, 4, 2, 0, 0, 1] and x[:, -1].tolist() == [15, 14, 12, 10, 10, 11]
    assert all(bool((x[i, :-1] == x[i, 0]).all()) for i in range(6))


def test_reorder_graph_and_stream(cuda_lib):
    x = torch.randn(8, 300, device="cuda")
    parents = torch.tensor([[1, 0, 3, 3], [0, 0, 0, 1]], device="cuda")
    want = _reordered(x, parents)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, = cuda_lib.beam_reorder(x, parents)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.beam_reorder(x, parents, out=x)
    count = x._version
    for _ in range(3):
        want = _reordered(x, parents)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    cuda_lib.beam_reorder(x, parents, out=x)
    assert x._version == count + 1


def test_reorder_refusals(cuda_lib):
    x = torch.randn(8, 10, device="cuda")
    p = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    with pytest.raises(cuda_lib.PstatError):  # the same memory twice
        cuda_lib.beam_reorder([x, x], p, out=[x, x])
    with pytest.raises(cuda_lib.PstatError):  # overlapping by a part of it
        store = torch.randn(20, 10, device="cuda")
        cuda_lib.beam_reorder([store[:8]], p, out=[store[4:12]])
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_reorder([x], p, out=[torch.zeros(10, device="cuda").expand(8, 10)])
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_reorder([torch.randn(130, 2, device="cuda")], p[:1])
    for args, out in (([], None), ([x.cpu()], None), ([x[:7]], None), ([x], [x[:4]]), ([x], [x.double()]),
                      ([x], [x, x]), ([torch.zeros(2, 1100, 3, 2, device="cuda")[:, :, :2, :1]], None)):
        with pytest.raises(ValueError):
            cuda_lib.beam_reorder(args, p, out=out)
    with pytest.raises(ValueError):
        cuda_lib.beam_reorder([x], p.int())
    with pytest.raises(ValueError):
        cuda_lib.beam_reorder([x], p.view(-1))
    # keys and values that take turns in one buffer are no overlap
    kv = torch.randn(8, 2, 5, 6, device="cuda")
    want = _reordered(kv, p)
    cuda_lib.beam_reorder([kv[:, 0], kv[:, 1]], p, out=[a := kv[:, 0], b := kv[:, 1]])
    assert torch.equal(kv, want) and a.data_ptr() != b.data_ptr()
