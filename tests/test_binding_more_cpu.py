"""The native module's optimiser, 8-bit head and beam search functions answer None, and raise
nothing, on whatever they do not take."""
import pytest
import torch

from test_binding_cpu import ODD, native


@pytest.mark.parametrize("x", range(len(ODD)))
def test_odd_tensors_are_not_taken(x):
    z = ODD[x]
    f = torch.zeros(3)
    assert native.adamw_step((z,), (z,), (z,), (z,), 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, None,
                             None, None) is None
    assert native.adamw_step((f,), (f,), (f,), (f,), 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, z, 1.0, None,
                             None) is None
    assert native.adamw_moments((z,), (z,), (z,), (z,), (z,)) is None
    assert native.fp8_quantize(z, 1, None) is None
    assert native.fp8_logits(z, z, z, z, True, None) is None
    assert native.beam_select(z, torch.zeros(1, 3), 4, None) is None
    assert native.beam_select(torch.zeros(3, 4), z, 4, None) is None
    assert native.beam_reorder((z,), torch.zeros(1, 3, dtype=torch.int64), None, None) is None
    assert native.beam_reorder((torch.zeros(3, 4),), z, None, None) is None


def test_counts_and_kinds():
    for f in (native.adamw_step, native.adamw_moments, native.fp8_quantize, native.fp8_logits,
              native.beam_select, native.beam_reorder):
        assert f() is None and f(1) is None
    for lists in ((), [], None, 3):
        assert native.adamw_step(lists, lists, lists, lists, 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, None,
                                 None, None, None) is None
        assert native.beam_reorder(lists, None, None, None) is None
    with pytest.raises(TypeError):
        native.bind_more()
    with pytest.raises(ValueError):
        native.bind_more(*[0] * 7)
