"""The fixed-point weights that draws and cuts are decided by, against exact values.

The bound.  With u = 2^-24, y = (M - z) log2(e)/t in double-float arithmetic:
the scale's low part is off by 2.75 u^2 (a residual and a constant, added, divided),
and y's low part, at most 3.25 u y, is formed with four roundings or dropped products
of 1, 2.25, 3.25 and 1.25 u^2 y: together 10.5 u^2 y, which is 10.5 x 2^-48 |x| of the
weight, below 2^-44.5 |x|.  The rest does not grow with x: the cubic and higher terms
of e^-s, s <= 2^-7.5, are at most 2^-25 with five roundings of u (2^-46.7), the low
word of the result, below 2^-24, takes one more (2^-48.6), tables and products are
below 2^-49, all relative to a mantissa of at least 1/2: 2^-45.  Rounding to k digits
adds half of the last one."""
import ctypes
import decimal
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(cuda_lib, tmp_path_factory):
    from vocab_wide_token_gb300 import build

    out = str(tmp_path_factory.mktemp("probe") / "probe.so")
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, f"-I{build.CSRC}", "-shared",
                        "-cudart", "shared", os.path.join(HERE, "fixed_weights_probe.cu"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    lib.fixed_weights_probe.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int, ctypes.c_void_p,
                                                                ctypes.c_int]

    def run(z, M, t, k):
        z, M, t = (torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda() for a in (z, M, t))
        w = torch.zeros(len(z), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        assert lib.fixed_weights_probe(z.data_ptr(), M.data_ptr(), t.data_ptr(), k, w.data_ptr(),
                                       len(z)) == 0
        return [int(x) for x in w.cpu()]

    return run


def _exact(z, M, t, k, ctx):
    x = ctx.divide(ctx.subtract(decimal.Decimal(float(z)), decimal.Decimal(float(M))),
                   decimal.Decimal(float(t)))
    return x, ctx.multiply(ctx.exp(x), decimal.Decimal(2) ** k)


@pytest.mark.parametrize("t", [1.0, 0.7, 1.3, 0.05, 2.0**-20, 2.0**20, 7e-4])
@pytest.mark.parametrize("top", [0.0, 3.7, 21.3, -0.013, 1500.25])
@pytest.mark.parametrize("k", [60, 52, 41])
def test_error_bound(probe, t, top, k):
    rng = np.random.default_rng(int(top * 8) + k + 1000)
    n = 600
    t32 = np.float32(t)
    x = np.concatenate([rng.uniform(0, 1, n), rng.uniform(0, k * 0.7, 2 * n), 10.0 ** rng.uniform(-9, 0, n)])
    M = np.full(len(x), np.float32(top), np.float32)
    z = np.minimum((np.float64(M[0]) - x * np.float64(t32)).astype(np.float32), M)
    got = probe(z, M, np.full(len(x), t32), k)
    ctx = decimal.Context(prec=60)
    for i, w in enumerate(got):
        xi, e = _exact(z[i], M[i], t32, k, ctx)
        bound = float(e) * (2.0**-45 + 2.0**-44.5 * abs(float(xi))) + 0.5
        assert abs(float(w - e)) <= bound * (1 + 1e-9), (i, float(xi), w, float(e))


def test_special_values(probe):
    M = np.float32([1.5, 1.5, 0.0, 0.0, 3e38, 3e38, -2.0])
    z = np.float32([1.5, -np.inf, -0.0, -1e-45, -3e38, 3e38, -2.0])
    t = np.float32([0.3, 1.0, 1.0, 1.0, 1.0, 2.0**-20, 2.0**20])
    for k in (41, 60):
        assert probe(z, M, t, k) == [2**k, 0, 2**k, 2**k, 0, 2**k, 2**k]
