"""The native marshalling module answers None, and raises nothing, on whatever it
does not take; the functions of pstat then refuse with their own errors."""
import pytest
import torch

from vocab_wide_token_gb300 import pstat

native = pytest.importorskip("vocab_wide_token_gb300._binding")

ODD = [
    None, 1, "x", [], torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.float64), torch.zeros(4),
    torch.zeros(3, 4, device="meta"), torch.zeros(3, 4).to_sparse(), torch.zeros(4, 3).t(),
    torch.zeros(0, 4), torch.quantize_per_tensor(torch.zeros(3, 4), 1.0, 0, torch.qint8),
]


@pytest.mark.parametrize("x", range(len(ODD)))
def test_odd_logits_are_not_taken(x):
    z = ODD[x]
    assert native.sample(z, torch.zeros(3), 1.0, 0, 1.0, 0.0, None) is None
    assert native.filtered_forward(z, None, 1.0, 0, 1.0, 0.0, -100, None) is None
    assert native.filtered_backward(z, None, None, torch.zeros(3, 2), torch.zeros(3),
                                    torch.zeros(3, dtype=torch.int64), 1.0, -100, None) is None
    assert native.grad_norm([z], None) is None
    assert native.clip_grad_norm([z], 1.0, None, None) is None
    assert native.clip_grad_norm([torch.zeros(2)], 1.0, [z], None) is None


def test_other_lists_and_counts_are_not_taken():
    for tensors in ([], (), None, {}, torch.zeros(3), iter([torch.zeros(3)]), [1], [None]):
        assert native.grad_norm(tensors, None) is None
        assert native.clip_grad_norm(tensors, 1.0, None, None) is None
    assert native.sample() is None
    assert native.filtered_forward(1) is None
    assert native.filtered_backward(1, 2) is None
    assert native.grad_norm() is None
    assert native.clip_grad_norm([torch.zeros(3)], "1", None, None) is None
    with pytest.raises(TypeError):
        native.bind()
    with pytest.raises(ValueError):
        native.bind(*[0] * 7)


def test_refusals_are_those_of_the_functions():
    z, u = torch.zeros(3, 4), torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        pstat.sample(z, u)
    with pytest.raises(ValueError, match="CUDA"):
        pstat.filtered_forward(z, None)
    with pytest.raises(ValueError, match="CUDA"):
        pstat.clip_grad_norm([u], 1.0)
    with pytest.raises(ValueError, match="empty"):
        pstat.grad_norm([])


def test_a_failed_launch_raises():
    assert pstat._launched((1,), "x") == (1,)
    with pytest.raises(pstat.PstatError, match="pstat_sample"):
        pstat._launched(-7, "pstat_sample")
