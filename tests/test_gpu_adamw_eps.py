"""The AdamW step's divisor sqrt(v) / sqrt(1 - b2^t) + eps over the range of eps, with squares of
gradients around and below the least normal fp32 number.

Moments and parameters are held to what test_gpu_adamw.py derives: v as an fp32 number is exact
(its code is the oracle's), so a root of one below 2^-126 has the error of any other.  eps
is rounded to fp32 once, which the 16 units of the update cover."""
import numpy as np
import pytest
import torch

from test_gpu_adamw import BF16, F32, _check, _expect

pytestmark = pytest.mark.gpu
EPS = [0.0, float(np.float32(1e-40)), 1e-30, 2.0**-60, 2.0**-59, 1e-17, 1e-15, 1e-12, 1e-8]


def _tiny(n, seed, p_type, g_type, bits, lib, lo, hi):
    """Gradients of 10^lo to 10^hi, a part of them zero, and fresh moments."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(n, generator=gen, dtype=torch.float64, device="cuda")
    sign = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0).double()
    g = (sign * 10.0 ** (lo + (hi - lo) * u)).to(g_type)
    p = (1e-3 * torch.randn(n, generator=gen, device="cuda")).to(p_type)
    return p, g, *lib.adamw_state(p, bits)


def _steps(lib, p, g, m, v, bits, eps, steps, seed, on_device=False):
    hyper = dict(betas=(0.9, 0.999), eps=eps, weight_decay=0.01)
    for step in steps:
        old = p.clone()
        want = _expect(p, g, m, v, bits, seed, 0, step, 1e-2, 1.0, **hyper)
        at = torch.tensor(step, device="cuda") if on_device else step
        lib.adamw_step([p], [g], [m], [v], at, 1e-2, **hyper, seed=seed)
        _check(p, old, m, v, want, bits, seed is not None)


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type,seed", [(F32, F32, None), (F32, BF16, 5), (BF16, BF16, None)])
def test_small_squares(cuda_lib, eps, bits, p_type, g_type, seed):
    """(1 - b2) g^2 from 1e-43 to 1e-33, at the first step, where the root is divided by
    sqrt(0.001), at the second and at a late one."""
    p, g, m, v = _tiny(2125, 1, p_type, g_type, bits, cuda_lib, -20, -15)
    _steps(cuda_lib, p, g, m, v, bits, eps, (1, 2, 5000), seed)


@pytest.mark.parametrize("eps", [1e-17, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_on_the_device(cuda_lib, eps, bits):
    p, g, m, v = _tiny(2125, 2, F32, F32, bits, cuda_lib, -20, -15)
    _steps(cuda_lib, p, g, m, v, bits, eps, (1, 40), 3, on_device=True)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [float(np.float32(1e-40)), 1e-30])
def test_squares_of_zero(cuda_lib, bits, eps):
    """g^2 below every fp32 number: the divisor is eps."""
    p, g, m, v = _tiny(2125, 3, F32, F32, bits, cuda_lib, -30, -24)
    _steps(cuda_lib, p, g, m, v, bits, eps, (1, 2), None)
    assert not bool(v[:2125].any())


@pytest.mark.parametrize("seed", [None, 3])
@pytest.mark.parametrize("eps", [1e-8, 1e-15, 1e-17])
def test_parameters_at_the_ends(cuda_lib, seed, eps):
    """Zeros, subnormals and large numbers in a block of codes, all finite; zeros in most of
    the others."""
    n = 1024
    g = torch.zeros(n, device="cuda")
    g[:5] = torch.tensor([0.0, 1e-45, 1e-30, 1e18, -1e18])
    g[128:136] = torch.tensor([1e-42, -1e-42, 1e-45, 3e-39, 0, 0, 1e-38, 1e-22])
    g[300:304] = torch.tensor([1e-18, -3.4e-18, 1e-20, 1.0])
    g[512] = -2e-18
    p = torch.ones(n, device="cuda")
    m, v = cuda_lib.adamw_state(p, 8)
    _steps(cuda_lib, p, g, m, v, 8, eps, (1, 2), seed)


@pytest.mark.parametrize("eps", [1e-15, 1e-17])
def test_the_same_bits_in_any_place(cuda_lib, eps):
    """Tensors on and off 16 bytes, whose blocks take different ways."""
    n = 200_077
    p, g, m, v = _tiny(n, 4, BF16, F32, 8, cuda_lib, -19, -12)
    results = []
    for off in (0, 1):
        got = []
        for x in (p, g, m, v):
            got.append(torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")[off:].copy_(x))
        for step in (1, 2, 3):
            cuda_lib.adamw_step([got[0]], [got[1]], [got[2]], [got[3]], step, 1e-2, eps=eps, seed=step)
        results.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*results))
