"""What a call writes into tensors of the caller's counts as an in-place change, so
that autograd notices when a tensor that it saved was overwritten."""
import pytest
import torch

from vocab_wide_token_gb300 import pstat

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "python"])
def path(request, cuda_lib, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(pstat, "_native", None)
    elif pstat._native is None:
        pytest.skip("the native module is not built")


@pytest.mark.parametrize("count", [1, 40])
def test_clipping_a_saved_tensor_is_noticed(path, count):
    a = [torch.randn(100, device="cuda", requires_grad=True) for _ in range(count)]
    b = [x.exp() for x in a]  # each saves its result
    pstat.clip_grad_norm([x.detach() for x in b], 1e-3)
    with pytest.raises(RuntimeError, match="inplace operation"):
        sum(x.sum() for x in b).backward()


def test_clipping_elsewhere_leaves_its_inputs_alone(path):
    a = torch.randn(100, device="cuda", requires_grad=True)
    b, out = a.exp(), torch.empty(100, device="cuda")
    seen = out._version
    pstat.clip_grad_norm([b.detach()], 1e-3, out=[out])
    assert out._version > seen
    pstat.grad_norm([b.detach()])
    b.sum().backward()
    assert torch.equal(a.grad, b.detach())


def test_outputs_given_to_the_other_calls(path):
    T, V = 3, 50
    z, u = torch.randn(T, V, device="cuda"), torch.rand(T, device="cuda")
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")
    drawn = (y.clone(), f(T))
    stats = (f(T), f(T), f(T, 2), f(T), y.clone())
    grad, norm = f(T, V), f()
    given = (*drawn, *stats, grad, norm)
    seen = [x._version for x in given]
    pstat.sample(z, u, out=drawn)
    pstat.filtered_forward(z, y, out=stats)
    pstat.filtered_backward(z, y, None, *stats[2:], out=grad)
    pstat.grad_norm([grad], out=norm)
    assert all(x._version > v for x, v in zip(given, seen))


def test_inference_tensors(path):
    """They have no counter, and are clipped all the same."""
    with torch.inference_mode():
        g = torch.full((100,), 1.0, device="cuda")
    norm, got = pstat.clip_grad_norm([g], 1.0)
    assert norm.item() == 10.0 and got[0] is g and abs(g[0].item() - 0.1) < 1e-8
    with torch.inference_mode():
        pstat.clip_grad_norm([g], 0.5)
    assert abs(g[0].item() - 0.05) < 1e-8
