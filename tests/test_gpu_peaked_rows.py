"""Rows without filters whose mass lies almost all on one token, S = 1 + X with a
small X: ln S, the label's logprob and its gradient (w/t) X / (1 + X) have to keep
the relative precision of X.

Tolerance.  Below S = 1 + 2^-6, X is a sum of exponentials of fp32 exponents: each
has 4 units of 2^-24 from ex2.approx and, with |a| <= 48 binary orders, two
roundings of a worth |a| ln 2 units each and as much from the rounded scale (100 in
all), and the sums of 8, 32 and 16 terms 8 + 5 + 16; the other chunks' share is
within 2^-18 (64 units); log1p, expm1 and the products add a dozen: below 2^8 units,
2^-16.  From 1 + 2^-6 on, S itself is within 2^-18, which is 2^-12 of X.  2^-12 holds
for both.  A bf16 gradient is rounded besides, half a step."""
import math

import numpy as np
import pytest
import torch

from helpers import to_oracle
from oracle import filters as oflt

pytestmark = pytest.mark.gpu
IGN = -100
BF16, F32 = torch.bfloat16, torch.float32
TOL = 2.0**-12


def _peaked(V, dtype, excess, tops, t, seed, pad=0, off=0):
    """Rows with their maximum in column tops[i] and about that excess on the others."""
    T = len(excess)
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, V, generator=g, device="cuda").clamp_(-3, 3)
    for i, x in enumerate(excess):
        z[i] = t * (z[i] + math.log(x / max(1, V - 1)) - 0.5) + 3.0
        z[i, tops[i]] = 3.0
    store = torch.full((off + T * (V + pad),), math.nan, device="cuda", dtype=dtype)
    return store.as_strided((T, V), (V + pad, 1), off).copy_(z)


def _excess(z, t):
    """X of every row, in float64 from the rounded logits."""
    t = float(np.float32(t))
    out = []
    for row in to_oracle(z.contiguous()):
        row = oflt.to_double(row)
        top = int(np.argmax(row))
        e = np.exp((row - row[top]) / t)
        e[top] = 0.0
        out.append(math.fsum(e))
    return np.array(out)


EXCESS = [0.5, 0.05, 2.0**-6, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 3e-7, 1e-7, 3e-8, 1e-9, 1e-11]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("V", [2, 33, 2049, 4097, 20011, 151936])
@pytest.mark.parametrize("t", [1.0, 0.6])
def test_statistics_and_gradient(cuda_lib, dtype, out_dtype, V, t):
    T = len(EXCESS)
    tops = [(i * 7919) % V for i in range(T)]
    tops[1], tops[2] = V - 1, 0
    for pad, off in ((0, 0), (1, 3)):
        z = _peaked(V, dtype, EXCESS, tops, t, V, pad, off)
        y = torch.tensor(tops, device="cuda")
        w = torch.linspace(-1.5, 2.0, T, device="cuda")
        lp, ent, rs, tau, idx = cuda_lib.filtered_forward(z, y, t)
        grad = cuda_lib.filtered_backward(z, y, w, rs, tau, idx, t, out_dtype=out_dtype)
        X = _excess(z, t)
        want = np.log1p(X)
        assert np.all(np.abs(rs[:, 1].double().cpu().numpy() - want) <= TOL * want), V
        assert np.all(np.abs(lp.double().cpu().numpy() + want) <= TOL * want), V
        got = grad.double().gather(1, y[:, None])[:, 0].cpu().numpy()
        want = w.double().cpu().numpy() / float(np.float32(t)) * X / (1 + X)
        step = 2.0**-8 if out_dtype == BF16 else 0.0
        assert np.all(np.abs(got - want) <= (TOL + step) * np.abs(want)), (V, got / want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [33, 5000, 151936])
def test_draws_by_every_kernel(cuda_lib, dtype, V):
    """The same logprob, bit for bit, whether the finish kernel decides the draw or
    (at u = 0, where no error bound does) the exact one, in batches of any size
    and next to rows with filters."""
    T = len(EXCESS)
    z = _peaked(V, dtype, EXCESS, [0] * T, 0.8, 5)
    stats = cuda_lib.filtered_forward(z, torch.zeros(T, dtype=torch.int64, device="cuda"), 0.8)
    want = np.log1p(_excess(z, 0.8))
    for u in (0.0, 0.25):
        tok, lp = cuda_lib.sample(z, torch.full((T,), u, device="cuda"), 0.8)
        assert bool((tok == 0).all()) and torch.equal(lp, stats[0])
        assert np.all(np.abs(lp.double().cpu().numpy() + want) <= TOL * want)
        k = torch.zeros(T * 50, dtype=torch.int32, device="cuda")
        k[1::2] = 5
        for n in (1, 24, 50):
            many = z.repeat(n, 1)
            us = torch.full((T * n,), u, device="cuda")
            tok2, lp2 = cuda_lib.sample(many, us, 0.8)
            assert torch.equal(lp2, lp.repeat(n)) and bool((tok2 == 0).all())
            _, lp3 = cuda_lib.sample(many, us, 0.8, k[:T * n].contiguous())
            assert torch.equal(lp3[::2], lp.repeat(n)[::2])
