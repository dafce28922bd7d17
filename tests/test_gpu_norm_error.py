"""The relative error of the gradient norm, bounded by its roundings.

A thread squares and adds its part of a unit of 32 KB in fp32, in four sums: 8
vectors of 16 bytes, so 8 fp32 squares to a sum, each added with one rounding, or
16 bf16 squares, which are exact (8 bits times 8), so that 15 additions round.
Joining the four sums takes two more.  Every term is positive, hence each rounding
is at most 2^-24 of the sum: 10 x 2^-24 (fp32) and 17 x 2^-24 (bf16).  All further
sums and the root are in fp64; the root halves the error, and the result is
rounded to fp32 once: 6 x 2^-24 and 9.5 x 2^-24."""
import pytest
import torch

from helpers import to_oracle
from oracle import filters as oflt

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BOUND = {F32: 6.001 * 2.0**-24, BF16: 9.501 * 2.0**-24}


def _rounded_up_each_time(units, dtype):
    """Each of the four sums starts at 1 and then takes squares just above half a
    step of 1, all of which round up."""
    per = 32768 // (2 if dtype == BF16 else 4)
    x = torch.full((units, per), 2.0**-12 * (1 + 2.0**-7), device="cuda")
    first = x[:, :2048] if dtype == BF16 else x[:, :1024]
    first.view(units, 256, -1)[:, :, :4] = 1.0
    return x.reshape(-1).to(dtype)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("units", [1, 16, 17, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_error_bound(cuda_lib, dtype, units, off):
    n = units * 32768 // (2 if dtype == BF16 else 4)
    g = torch.Generator(device="cuda").manual_seed(units)
    inputs = {
        "up": _rounded_up_each_time(units, dtype),
        "constant": torch.full((n,), 0.3, device="cuda").to(dtype),
        "random": torch.randn(n, generator=g, device="cuda").to(dtype),
        "wide": (torch.randn(n, generator=g, device="cuda")
                 * 10.0 ** (-6 * torch.rand(n, generator=g, device="cuda"))).to(dtype),
    }
    for name, x in inputs.items():
        store = torch.empty(n + off, device="cuda", dtype=dtype)
        view = store[off:].copy_(x)
        want = oflt.grad_norm([to_oracle(x)])
        got = cuda_lib.grad_norm([view]).item()
        assert abs(got - want) <= BOUND[dtype] * want, (name, (got - want) / want * 2**24)
