"""Clipping whose factor max_norm / norm lies below the least normal fp32 number.

The scaled elements are ordinary numbers (about max_norm / sqrt(n)), so they have
the error of any other clipping: the norm's (at most 9 x 2^-24, test_gpu_norm_error.py),
the factor's and the product's roundings (2^-24 each) and the one to the output's
type, half a step."""
import pytest
import torch

from helpers import to_oracle
from oracle import filters as oflt

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e-8, 1e-20, 1e-30])
@pytest.mark.parametrize("sizes", [[5000], [5000, 33], [300001, 7]], ids=str)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_factors_below_the_normal_numbers(cuda_lib, dtype, off, sizes, limit):
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [(1e36 / n**0.5 * 60 * torch.randn(n + off, generator=g, device="cuda")).to(dtype)[off:]
          for n in sizes]
    want = oflt.grad_norm([to_oracle(x) for x in xs])
    assert 1e37 < want < 3e38
    limit = torch.tensor(limit, dtype=torch.float32).item()
    outs = [torch.empty_like(x) for x in xs]
    err = cuda_lib.new_error_flag("cuda:0")
    norm, _ = cuda_lib.clip_grad_norm(xs, limit, out=outs, dev_error=err)
    assert err.item() == 0 and abs(norm.item() - want) <= 10 * 2.0**-24 * want
    step = 2.0**-8 if dtype == BF16 else 2.0**-24
    for x, o in zip(xs, outs):
        exact = x.double() * (limit / want)
        # below 2^-126 numbers are spaced 2^-149, in bf16 2^-133
        tiny = 2.0**-133 if dtype == BF16 else 2.0**-149
        assert bool(((o.double() - exact).abs()
                     <= (step + 11 * 2.0**-24) * exact.abs() + tiny).all())
    own = [x.clone() for x in xs]
    cuda_lib.clip_grad_norm(own, limit)
    assert all(torch.equal(a, b) for a, b in zip(own, outs))
