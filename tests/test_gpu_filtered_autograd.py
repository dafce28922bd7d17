"""The gradient of filtered_policy_stats has no derivative of its own here: asking
for one raises, and does not take it for a constant."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_second_derivative_raises(cuda_lib):
    z = torch.randn(4, 300, device="cuda", requires_grad=True)
    y = torch.tensor([0, 5, 7, 299], device="cuda")
    lp, _ = cuda_lib.filtered_policy_stats(z, y, 0.9)
    (g,) = torch.autograd.grad(lp.sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        (g.square().sum() + z.square().sum()).backward()


def test_first_derivative_next_to_other_terms(cuda_lib):
    z = torch.randn(4, 300, device="cuda", requires_grad=True)
    y = torch.tensor([0, 5, 7, 299], device="cuda")

    def loss():
        return cuda_lib.filtered_policy_stats(z, y, 0.9, 0, 0.95)[0].sum() + z.square().sum()

    (plain,) = torch.autograd.grad(loss(), z)
    (kept,) = torch.autograd.grad(loss(), z, create_graph=True)
    assert torch.equal(plain, kept)
    lp, _ = cuda_lib.filtered_policy_stats(z, y, 0.9, 0, 0.95)
    (alone,) = torch.autograd.grad(lp.sum(), z)
    assert torch.allclose(plain, alone + 2 * z.detach(), rtol=1e-6, atol=1e-6)


def test_second_derivative_through_the_incoming_gradient(cuda_lib):
    z = torch.randn(4, 300, device="cuda", requires_grad=True)
    y = torch.tensor([0, 5, 7, 299], device="cuda")
    v = torch.ones(4, device="cuda", requires_grad=True)
    lp, _ = cuda_lib.filtered_policy_stats(z, y, torch.full((4,), 0.9, device="cuda"))
    (g,) = torch.autograd.grad(lp, z, v, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        g.square().sum().backward()
