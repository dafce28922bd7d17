"""Global gradient norm and clipping against the float64 oracle.

The sum of squares is accumulated in fp64 from fp32 sums of at most 8 squares
(8 roundings of 2^-24 relative, halved by the square root), and the result is
rounded to fp32 once: 5 x 2^-24 relative covers it.  The factor and the product
are rounded to fp32 once each and the result once to the output's type."""
import math

import numpy as np
import pytest
import torch

from helpers import to_oracle
from oracle import filters as oflt

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _list(sizes, seed, dtypes=(BF16, F32), scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def _norm(xs):
    return oflt.grad_norm([to_oracle(x) for x in xs])


LISTS = [[1], [0], [3, 0, 5], [1, 2, 3, 7, 8, 9, 15, 16, 17, 4095, 4097, 8191, 8193],
         [100003, 5, 65536, 1], list(range(1, 70)), [17] * 900, [2000003]]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(cuda_lib, sizes):
    xs = _list(sizes, len(sizes))
    want = _norm(xs)
    got = cuda_lib.grad_norm(xs)
    assert abs(got.item() - want) <= 5 * 2.0**-24 * want
    for share in (0.25, 4.0):
        limit = share * want if want else 1.0
        outs = [torch.empty_like(x) for x in xs]
        keep = [x.clone() for x in xs]
        norm, res = cuda_lib.clip_grad_norm(xs, limit, out=outs)
        assert torch.equal(norm, got) and all(a is b for a, b in zip(res, outs))
        factor = min(1.0, limit / want) if want else 1.0
        for x, k, o in zip(xs, keep, outs):
            assert torch.equal(x, k)
            exact = k.double() * factor
            step = 2.0**-8 if k.dtype == BF16 else 2.0**-24
            assert bool(((o.double() - exact).abs() <= (step + 8 * 2.0**-24) * exact.abs()).all())
        norm2, res2 = cuda_lib.clip_grad_norm(xs, limit)
        for x, o in zip(xs, outs):
            assert torch.equal(x, o)  # in place: the same bits
        xs = keep


def test_unaligned_and_repeated(cuda_lib):
    base = _list([5000], 3)[0]
    base32 = base.float()
    xs = [base[1:4000], base32[3:], base[4001:]]
    want = _norm(xs)
    got = cuda_lib.grad_norm(xs)
    assert abs(got.item() - want) <= 5 * 2.0**-24 * want
    for _ in range(3):
        assert torch.equal(cuda_lib.grad_norm(xs), got)
    # the same tensor twice counts twice in the norm
    twice = cuda_lib.grad_norm([base32, base32])
    assert abs(twice.item() - math.sqrt(2) * _norm([base32])) <= 8 * 2.0**-24 * twice.item()
    for bad in ([base32, base32], [base32[:100], base32[50:]]):
        with pytest.raises(cuda_lib.PstatError):
            cuda_lib.clip_grad_norm(bad, 1.0)
    guard = torch.full((4096,), 5.0, device="cuda")
    cuda_lib.clip_grad_norm([guard[7:4000]], 1.0)
    assert bool((guard[:7] == 5).all()) and bool((guard[4000:] == 5).all())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e18, 1e25, 1e33])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_range(cuda_lib, scale, dtype):
    """Values whose squares leave fp32."""
    xs = _list([30011, 7], 5, (dtype,), scale)
    want = _norm(xs)
    got = cuda_lib.grad_norm(xs).item()
    # a subnormal result is spaced 2^-149
    assert abs(got - want) <= 5 * 2.0**-24 * want + 2.0**-149
    norm, res = cuda_lib.clip_grad_norm(xs, 1.0)
    if want > 1:
        assert abs(_norm(res) - 1.0) <= 2.0**-7


def test_zero_and_nonfinite(cuda_lib):
    zero = [torch.zeros(1000, device="cuda")]
    err = cuda_lib.new_error_flag("cuda:0")
    assert cuda_lib.grad_norm(zero, dev_error=err).item() == 0.0
    norm, res = cuda_lib.clip_grad_norm(zero, 1.0, dev_error=err)
    assert err.item() == 0 and bool((res[0] == 0).all())
    for bad in (math.nan, math.inf, -math.inf):
        xs = _list([4000, 33], 6)
        xs[1][5] = bad
        keep = [x.clone() for x in xs]
        err.zero_()
        assert not math.isfinite(cuda_lib.grad_norm(xs, dev_error=err).item())
        assert err.item() == cuda_lib.DEV_NONFINITE
        err.zero_()
        outs = [torch.empty_like(x) for x in xs]
        norm, _ = cuda_lib.clip_grad_norm(xs, 1.0, out=outs, dev_error=err)
        assert err.item() == cuda_lib.DEV_NONFINITE and not math.isfinite(norm.item())
        for o, k in zip(outs, keep):
            assert torch.equal(o.view(torch.int16 if o.dtype == BF16 else torch.int32),
                               k.view(torch.int16 if k.dtype == BF16 else torch.int32))
    # max_norm 0 zeroes a finite list
    xs = _list([100], 8)
    norm, res = cuda_lib.clip_grad_norm(xs, 0.0)
    assert bool((res[0] == 0).all())


def test_graph_and_lmhead_gradients(cuda_lib):
    """The lm_head backward's own gradients, clipped in a captured graph."""
    T, V, d = 130, 700, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    W = (0.1 * torch.randn(V, d, generator=g, device="cuda")).to(BF16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    lp, ent, rs = cuda_lib.lmhead_forward(h, W, y)
    dh, dW = cuda_lib.lmhead_backward(h, W, y, torch.randn(T, generator=g, device="cuda"), rs)
    outs = [torch.empty_like(dh), torch.empty_like(dW)]
    cuda_lib.clip_grad_norm([dh, dW], 0.1, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = cuda_lib.clip_grad_norm([dh, dW], 0.1, out=outs)
    for k in range(2):
        dh.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = _norm([dh, dW])
        assert abs(norm.item() - want) <= 5 * 2.0**-24 * want
        assert abs(_norm(outs) - min(0.1, want)) <= 8 * 2.0**-24


@pytest.mark.parametrize("units", [1, 2, 15, 16, 17, 40])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_launch_and_two(cuda_lib, dtype, units):
    """Lists on either side of 16 units of 32 KB, aligned or not, among empty
    tensors: norm, scaling, tiny and huge values, a NaN passed on."""
    per = 32768 // (2 if dtype == BF16 else 4)
    err = cuda_lib.new_error_flag("cuda:0")
    for off, scale in ((0, 1.0), (1, 1.0), (0, 1e-30), (3, 1e25)):
        store = _list([units * per + 8], units, (dtype,), scale)[0]
        whole = store[off:off + units * per - 5]
        cut = whole.numel() // 2 // per * per
        for xs in ([whole], [whole[:cut], whole[:0], whole[cut:]], [whole[:0]] * 40 + [whole]):
            want = _norm(xs)
            err.zero_()
            got = cuda_lib.grad_norm(xs, dev_error=err)
            assert abs(got.item() - want) <= 5 * 2.0**-24 * want + 2.0**-149
            limit = float(np.float32(want * 0.5))
            outs = [torch.empty_like(x) for x in xs]
            norm, _ = cuda_lib.clip_grad_norm(xs, limit, out=outs, dev_error=err)
            assert torch.equal(norm, got) and err.item() == 0
            step = 2.0**-8 if dtype == BF16 else 2.0**-24
            for x, o in zip(xs, outs):
                exact = x.double() * (limit / want if want > limit else 1.0)
                tiny = 2.0**-133 if dtype == BF16 else 2.0**-149  # subnormal results
                # the factor carries the norm's error and two roundings
                assert bool(((o.double() - exact).abs()
                             <= (step + 8 * 2.0**-24) * exact.abs() + tiny).all())
            own = [x.clone() for x in xs]
            cuda_lib.clip_grad_norm(own, limit)
            assert all(torch.equal(a, b) for a, b in zip(own, outs))
        keep = store.clone()
        whole[-1] = math.nan
        keep[off + units * per - 6] = math.nan
        norm, _ = cuda_lib.clip_grad_norm([whole], 1e-3, dev_error=err)
        assert math.isnan(norm.item()) and err.item() == cuda_lib.DEV_NONFINITE
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(store.view(bits), keep.view(bits))
