"""Steps and learning rates on the device: what is refused as a number sets DEV_BAD_PARAM there,
and changes nothing."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _state(lib, kinds):
    g = torch.Generator(device="cuda").manual_seed(1)
    ps, gs, ms, vs = [], [], [], []
    for i, (dtype, bits) in enumerate(kinds):
        ps.append(torch.randn(3000 + 77 * i, generator=g, device="cuda").to(dtype))
        gs.append(torch.randn(3000 + 77 * i, generator=g, device="cuda").to(dtype))
        m, v = lib.adamw_state(ps[-1], bits)
        ms.append(m)
        vs.append(v)
    lib.adamw_step(ps, gs, ms, vs, 1, 1e-2, seed=1)
    return ps, gs, ms, vs


BAD = [(0, 1e-3), (-1, 1e-3), (-(1 << 62), 1e-3), (5, -1e-3), (5, math.nan), (5, math.inf), (5, -math.inf), (0, math.nan)]


@pytest.mark.parametrize("step,lr", BAD)
@pytest.mark.parametrize("kinds", [[(F32, 32)], [(BF16, 8)], [(F32, 32), (BF16, 32), (F32, 8), (BF16, 8)]], ids=str)
def test_refused_on_the_device(cuda_lib, step, lr, kinds):
    ps, gs, ms, vs = _state(cuda_lib, kinds)
    before = [x.clone() for x in ps + ms + vs]
    at = torch.tensor(step, device="cuda")
    rate = torch.tensor(lr, dtype=F32, device="cuda")
    for a, b in ((at, rate), (at, 1e-3), (3, rate)):
        if not (step < 1 and a is at) and not (not 0 <= lr < math.inf and b is rate):
            continue  # what is left of the pair is no fault
        err = cuda_lib.new_error_flag("cuda:0")
        cuda_lib.adamw_step(ps, gs, ms, vs, a, b, seed=2, dev_error=err)
        assert err.item() == cuda_lib.DEV_BAD_PARAM
        assert all(torch.equal(x, y) for x, y in zip(before, ps + ms + vs))
    # beside a norm that is not finite: both bits
    err = cuda_lib.new_error_flag("cuda:0")
    cuda_lib.adamw_step(ps, gs, ms, vs, at, rate, norm=torch.tensor(math.nan, device="cuda"), max_norm=1.0,
                        dev_error=err)
    assert err.item() == cuda_lib.DEV_BAD_PARAM | cuda_lib.DEV_NONFINITE
    assert all(torch.equal(x, y) for x, y in zip(before, ps + ms + vs))


def test_replay_goes_on_after_a_refusal(cuda_lib):
    """A captured step skips a replay with a bad setting; rate 0 and step 1 are none."""
    ps, gs, ms, vs = _state(cuda_lib, [(F32, 32)])
    step, rate = torch.tensor(1, device="cuda"), torch.tensor(0.0, device="cuda")
    err = cuda_lib.new_error_flag("cuda:0")
    cuda_lib.adamw_step(ps, gs, ms, vs, step, rate, dev_error=err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.adamw_step(ps, gs, ms, vs, step, rate, dev_error=err)
    for s, r, want in ((2, 1e-3, 0), (0, 1e-3, cuda_lib.DEV_BAD_PARAM), (3, 1e-3, 0), (1, 0.0, 0),
                       (4, -1e-3, cuda_lib.DEV_BAD_PARAM)):
        step.fill_(s)
        rate.fill_(r)
        err.zero_()
        other = [[x.clone() for x in y] for y in (ps, ms, vs)]
        graph.replay()
        if not want:
            cuda_lib.adamw_step(other[0], gs, other[1], other[2], s, torch.tensor(r, dtype=F32).item())
        torch.cuda.synchronize()
        assert err.item() == want
        assert all(torch.equal(a, b) for x, y in zip(other, (ps, ms, vs)) for a, b in zip(x, y))
