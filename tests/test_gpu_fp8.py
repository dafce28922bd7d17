"""Quantising to e4m3 against a search among its values, and the 8-bit head's logits against
float64.

A code is rounded once, from an exact quotient: it has to be the oracle's.  A logit:
the tensor cores add 32 products to an accumulator at a time; taken as aligned to the
largest and cut at 2^-23 of it, 33 terms lose at most 33 x 2^-23 of it, four times in a
block: below 2^-15.9 of the block's sum of magnitudes.  The sum over blocks adds 2^-24 each
(at most 2^-18 for 64 blocks), the scale's product 2^-24, the output half a step."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _matrix(T, K, dtype, seed, pad=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.zeros(T * (K + pad) + off, dtype=dtype, device="cuda")
    x = store[off:].view(T, K + pad)[:, :K]
    x.copy_(torch.randn(T, K, generator=g, device="cuda") *
            torch.exp(3 * torch.randn(T, 1, generator=g, device="cuda")))
    return x


def _values(q):
    return q.float().double().cpu().numpy()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K,pad,off", [(1, 1, 0, 0), (3, 127, 1, 1), (128, 128, 0, 0), (130, 129, 0, 0),
                                         (257, 1000, 8, 0), (64, 384, 0, 8), (200, 260, 3, 5)])
def test_quantize(cuda_lib, rows, dtype, T, K, pad, off):
    x = _matrix(T, K, dtype, T + K, pad, off)
    x[T // 2, K // 2:] = 0
    err = cuda_lib.new_error_flag("cuda:0")
    q, s = cuda_lib.fp8_quantize(x, rows, dev_error=err)
    wq, ws = ofp8.quantize(x.double().cpu().numpy(), rows)
    assert err.item() == 0
    assert np.array_equal(s.double().cpu().numpy(), ws)
    assert np.array_equal(_values(q), wq)
    assert s.stride() == ((1, T) if rows == 1 and s.shape[1] > 1 and T > 1 else s.stride())
    if K > 1:
        # into given tensors, scales in either order
        for order in (torch.empty(ws.shape, device="cuda"), torch.empty(ws.shape[::-1], device="cuda").t()):
            out = torch.empty_like(q), order
            got = cuda_lib.fp8_quantize(x, rows, out=out)
            assert got[0] is out[0] and got[1] is out[1]
            assert torch.equal(out[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(out[1], s)


def test_quantize_range(cuda_lib):
    """Every tie and every border between two codes; the ends of fp32; what is not finite."""
    table = ofp8.e4m3_values()
    mid = (table[1:] + table[:-1]) / 2
    near = np.concatenate([table, mid, np.nextafter(mid.astype(np.float32), np.float32(np.inf)),
                           np.nextafter(mid.astype(np.float32), np.float32(0))])
    rows = []
    for e in (-126, -100, 0, 5, 118):
        for part in np.array_split(near, 8):
            row = np.zeros(128)
            row[:len(part)] = part * 2.0**e
            row[127] = 448.0 * 2.0**e
            rows.append(row)
    for top in (3.4e38, 448.0, np.nextafter(np.float32(448), np.float32(500)), 1e-45, 1e-38, 2.0**-126, 500.0):
        row = np.zeros(128)
        row[3], row[5] = -top, top / 3
        rows.append(row)
    x = torch.tensor(np.array(rows), dtype=F32, device="cuda")
    q, s = cuda_lib.fp8_quantize(x)
    wq, ws = ofp8.quantize(x.double().cpu().numpy(), 1)
    assert np.array_equal(s.double().cpu().numpy(), ws) and np.array_equal(_values(q), wq)
    for dtype in (BF16, F32):
        for rows in (1, 128):
            for bad in (math.nan, math.inf, -math.inf):
                x = _matrix(150, 300, dtype, 1)
                x[7, 140] = bad
                err = cuda_lib.new_error_flag("cuda:0")
                q, s = cuda_lib.fp8_quantize(x, rows, dev_error=err)
                assert err.item() == cuda_lib.DEV_NONFINITE
                wq, ws = ofp8.quantize(x.double().cpu().numpy(), rows)
                assert np.array_equal(s.double().cpu().numpy(), ws, equal_nan=True)
                assert np.array_equal(_values(q), wq)


def _head(T, V, K, seed, general=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, s = ((torch.randn(T, K, generator=g, device="cuda") * 60).clamp_(-448, 448).to(E4M3),
            torch.exp(torch.randn(-(-K // 128), T, generator=g, device="cuda")).t())
    W = (torch.randn(V, K, generator=g, device="cuda") * 60).clamp_(-448, 448).to(E4M3)
    Ws = torch.exp(torch.randn(-(-V // 128), -(-K // 128), generator=g, device="cuda"))
    if not general:
        s, Ws = torch.exp2(torch.round(s)), torch.exp2(torch.round(Ws))
    return q, s, W, Ws


def _exact(q, s, W, Ws):
    """(logits, sums of magnitudes) in float64."""
    T, K = q.shape
    V = W.shape[0]
    x = q.float().double() * s.double().repeat_interleave(128, 1)[:, :K]
    w = W.float().double() * Ws.double().repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :K]
    return x @ w.T, x.abs() @ w.abs().T


def _check(got, q, s, W, Ws):
    want, size = _exact(q, s, W, Ws)
    room = size * (2.0**-15.9 + 2.0**-18 + 2.0**-24) + want.abs() * (2.0**-8 if got.dtype == BF16 else 2.0**-24)
    off = (got.double() - want).abs()
    assert bool((off <= room).all()), (float((off / room).max()), int((off > room).sum()))
    return float((off / size.clamp_min(1e-300)).max())


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,V,K", [
    (1, 1, 16), (1, 300, 128), (5, 129, 144), (16, 1000, 256), (17, 128, 4096), (33, 257, 400), (64, 999, 1024),
    (65, 2000, 512), (128, 1001, 640), (129, 500, 512), (201, 20000, 256), (256, 300, 1040), (257, 513, 128),
    (600, 1111, 384), (1, 20001, 2048)])
def test_logits(cuda_lib, out, T, V, K):
    q, s, W, Ws = _head(T, V, K, T + V)
    err = cuda_lib.new_error_flag("cuda:0")
    got = cuda_lib.fp8_logits(q, s, W, Ws, out, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and got.dtype == out and got.shape == (T, V)
    _check(got, q, s, W, Ws)


def test_logits_are_nearly_those_of_fp32(cuda_lib):
    """The accumulators' error as it is, on sums without cancelled products: below 2^-20 of
    the magnitudes (the bound above is for all bits lost one way)."""
    q, s, W, Ws = _head(64, 2000, 4096, 2)
    assert _check(cuda_lib.fp8_logits(q, s, W, Ws, F32), q, s, W, Ws) <= 2.0**-20


def test_same_bits_in_any_batch(cuda_lib):
    """Row by row, through tiles of every width."""
    q, s, W, Ws = _head(700, 1500, 1024, 3)
    whole = cuda_lib.fp8_logits(q, s, W, Ws, F32)
    for lo, hi in ((0, 1), (5, 20), (20, 52), (100, 164), (200, 328), (300, 500), (0, 256), (37, 294), (699, 700)):
        part = cuda_lib.fp8_logits(q[lo:hi], s[lo:hi], W, Ws, F32)
        assert torch.equal(part, whole[lo:hi]), (lo, hi)
    again = cuda_lib.fp8_logits(q, s, W, Ws, F32)
    assert torch.equal(again, whole)


def test_outputs_strides_and_guards(cuda_lib):
    q, s, W, Ws = _head(70, 777, 256, 4)
    for dtype in (BF16, F32):
        want = cuda_lib.fp8_logits(q, s, W, Ws, dtype)
        store = torch.full((72, 800), 7.0, dtype=dtype, device="cuda")
        out = store[1:71, 3:780]
        assert cuda_lib.fp8_logits(q, s, W, Ws, out=out) is out
        assert torch.equal(out, want)
        store[1:71, 3:780] = 7
        assert bool((store == 7).all())
        # scales by rows
        assert torch.equal(cuda_lib.fp8_logits(q, s.contiguous(), W, Ws, dtype), want)


def test_a_scale_that_is_not_finite(cuda_lib):
    q, s, W, Ws = _head(40, 300, 512, 5)
    want = cuda_lib.fp8_logits(q, s, W, Ws, F32)
    s = s.clone()
    s[3, 1] = math.nan
    got = cuda_lib.fp8_logits(q, s, W, Ws, F32)
    assert bool(torch.isnan(got[3]).all())
    rest = [i for i in range(40) if i != 3]
    assert torch.equal(got[rest], want[rest])


def test_graph_and_stream(cuda_lib):
    q, s, W, Ws = _head(20, 3000, 512, 6)
    want = cuda_lib.fp8_logits(q, s, W, Ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cuda_lib.fp8_logits(q, s, W, Ws)
    side.synchronize()
    assert torch.equal(got, want)
    x = torch.randn(20, 512, device="cuda").to(BF16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = cuda_lib.fp8_quantize(x)
        got = cuda_lib.fp8_logits(a, b, W, Ws)
    for _ in range(2):
        x.mul_(1.7)
        graph.replay()
        torch.cuda.synchronize()
        c, d = cuda_lib.fp8_quantize(x)
        assert torch.equal(got, cuda_lib.fp8_logits(c, d, W, Ws))
    assert cuda_lib.fp8_logits(q[:0], s[:0], W, Ws).shape == (0, 3000)


def test_refusals(cuda_lib):
    q, s, W, Ws = _head(8, 300, 256, 7)
    for args in ((q.float(), s, W, Ws), (q, s, W.float(), Ws), (q, s[:4], W, Ws), (q, s.double(), W, Ws),
                 (q, s, W[:, :128], Ws), (q, s, W, Ws[:2]), (q, s, W, Ws.t()), (q.t(), s, W, Ws), (q, s, W.cpu(), Ws)):
        with pytest.raises(ValueError):
            cuda_lib.fp8_logits(*args)
    with pytest.raises(TypeError):
        cuda_lib.fp8_logits(q, s, W, Ws, torch.float16)
    with pytest.raises(ValueError):
        cuda_lib.fp8_logits(q, s, W, Ws, out=torch.empty(8, 301, device="cuda"))
    with pytest.raises(cuda_lib.PstatError):  # K not a multiple of 16
        cuda_lib.fp8_logits(torch.zeros(2, 24, device="cuda").to(E4M3), torch.ones(2, 1, device="cuda"),
                            torch.zeros(5, 24, device="cuda").to(E4M3), torch.ones(1, 1, device="cuda"))
    flat = torch.zeros(2 * 32 + 1, device="cuda").to(E4M3)
    with pytest.raises(cuda_lib.PstatError):  # off 16 bytes
        cuda_lib.fp8_logits(flat[1:].view(2, 32), torch.ones(2, 1, device="cuda"),
                            torch.zeros(5, 32, device="cuda").to(E4M3), torch.ones(1, 1, device="cuda"))
    x = torch.zeros(4, 100, device="cuda")
    for bad in (dict(rows=2), dict(out=(torch.empty(4, 100, device="cuda"), s))):
        with pytest.raises(ValueError):
            cuda_lib.fp8_quantize(x, **bad)
    with pytest.raises(TypeError):
        cuda_lib.fp8_quantize(x.half())
    with pytest.raises(ValueError):
        cuda_lib.fp8_quantize(x.cpu())
