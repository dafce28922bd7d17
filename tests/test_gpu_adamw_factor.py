"""The step on gradients so large that the factor max_norm / norm lies below the least normal
fp32 number, while the clipped gradients are ordinary ones.

The factor is one quotient, rounded to 24 bits; moments are the products and sums of
test_gpu_adamw.py from there, to the bit."""
import numpy as np
import pytest
import torch

from oracle import adamw as oadam
from test_gpu_adamw import BF16, F32, HYPER, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e-6, 1e-8, 1e-20])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type,off", [(F32, F32, 0), (BF16, BF16, 0), (F32, BF16, 1)])
def test_factors_below_the_normal_numbers(cuda_lib, limit, bits, p_type, g_type, off):
    n = 5000
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = (limit * torch.randn(n + off, generator=gen, device="cuda")).to(p_type)[off:]
    g = (2e36 * torch.randn(n + off, generator=gen, device="cuda")).to(g_type)[off:]
    m, v = cuda_lib.adamw_state(p, bits)
    norm = cuda_lib.grad_norm([g])
    limit = np.float32(limit)
    factor = limit.astype(np.float64) / float(norm.item())
    assert 1e38 < norm.item() < 2e38 and factor < 2.0**-126
    # the factor to 24 bits, whatever its exponent; its product to fp32
    lead, e = np.frexp(factor)
    factor = np.ldexp(np.round(lead * 2.0**24), int(e) - 24)
    clipped = (g.double().cpu().numpy() * factor).astype(np.float32)
    for step, seed in ((1, None), (2, 9)):
        old = p.clone()
        m0 = oadam.decode(m.cpu().numpy(), n, "m") if bits == 8 else m.cpu().numpy()
        v0 = oadam.decode(v.cpu().numpy(), n, "v") if bits == 8 else v.cpu().numpy()
        m1, v1 = oadam.moments(m0, v0, clipped, 1.0, 0.9, 0.999)
        exact = oadam.parameter(old.double().cpu().numpy(), m1, v1, step, 1e-3, 0.9, 0.999, 1e-8, 0.01)
        to_m, to_v, _ = oadam.draws(seed, 0, n)
        want = (exact, m1, v1) if bits == 32 else (exact, oadam.encode(m1, to_m, "m"), oadam.encode(v1, to_v, "v"))
        err = cuda_lib.new_error_flag("cuda:0")
        cuda_lib.adamw_step([p], [g], [m], [v], step, 1e-3, **HYPER, norm=norm, max_norm=float(limit),
                            seed=seed, dev_error=err)
        assert err.item() == 0
        _check(p, old, m, v, want, bits, seed is not None)
