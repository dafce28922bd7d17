"""The tensors of a gradient list stay alive, and are the ones returned, whatever
another thread does to the caller's list while the native module runs without
the interpreter lock.  A stand-in for the module changes the list at that point."""
import weakref

import pytest
import torch

from vocab_wide_token_gb300 import pstat


class Emptying:
    """Answers as the module does, after the caller's lists have been emptied."""

    def __init__(self, *lists):
        self.lists = lists
        self.alive = None

    def _run(self, tensors, outs):
        refs = [weakref.ref(x) for x in tensors] + [weakref.ref(x) for x in outs or ()]
        for x in self.lists:
            x.clear()
        self.alive = [r() is not None for r in refs]
        return torch.zeros(())

    def grad_norm(self, tensors, dev_error):
        return self._run(tensors, None)

    def clip_grad_norm(self, tensors, max_norm, out, dev_error):
        return self._run(tensors, out)


def test_norm_keeps_its_tensors(monkeypatch):
    g = [torch.zeros(n) for n in (3, 5, 7)]
    fake = Emptying(g)
    monkeypatch.setattr(pstat, "_native", fake)
    pstat.grad_norm(g)
    assert fake.alive == [True] * 3


@pytest.mark.parametrize("apart", [False, True])
def test_clipping_keeps_and_returns_its_tensors(monkeypatch, apart):
    g = [torch.zeros(n) for n in (3, 5, 7)]
    out = [torch.empty(n) for n in (3, 5, 7)] if apart else None
    fake = Emptying(*([g, out] if apart else [g]))
    monkeypatch.setattr(pstat, "_native", fake)
    _, got = pstat.clip_grad_norm(g, 1.0, out=out)
    assert fake.alive == [True] * (6 if apart else 3)
    assert isinstance(got, list) and [x.numel() for x in got] == [3, 5, 7]
