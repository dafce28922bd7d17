"""Both marshalling paths of the optimiser, 8-bit head and beam search calls give the same bits
and refuse the same."""
import pytest
import torch

from test_gpu_binding import both, same  # noqa: F401  (a fixture)
from vocab_wide_token_gb300 import pstat

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("seed", [None, 5, -1, 1 << 63])
def test_adamw(both, bits, seed):
    g = torch.Generator(device="cuda").manual_seed(1)
    ps = [torch.randn(n, generator=g, device="cuda").to(t) for n, t in ((5, F32), (300, BF16), (0, F32))]
    gs = [torch.randn(p.shape, generator=g, device="cuda").to(BF16) for p in ps]
    norm = pstat.grad_norm(gs)

    def call():
        p = [x.clone() for x in ps]
        m, v = (list(x) for x in zip(*(pstat.adamw_state(x, bits) for x in p)))
        counts = [x._version for x in p + m + v]
        got = pstat.adamw_step(p, gs, m, v, 1, 1e-2, seed=seed, norm=norm, max_norm=1.0)
        assert all(a is b for a, b in zip(got, p, strict=True))
        assert [x._version for x in p + m + v] == [c + 1 for c in counts]
        if bits == 32:
            return p + m + v
        out = [[torch.empty_like(x, dtype=F32) for x in p] for _ in range(2)]
        a, b = pstat.adamw_moments(m, v, p, out=out)
        c, d = pstat.adamw_moments(m, v, p)
        same(a + b, c + d)
        assert all(x is y for x, y in zip(a + b, out[0] + out[1], strict=True))
        return p + m + v + a + b

    same(*both(call))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head(both, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(5, 272, generator=g, device="cuda").to(dtype)[:, :256]
    W = torch.randn(300, 256, generator=g, device="cuda").to(dtype)
    for out in (BF16, F32):
        def call():
            q, s = pstat.fp8_quantize(x)
            w, ws = pstat.fp8_quantize(W, 128)
            assert s.stride() == (1, 5)
            return q, s, w, ws, pstat.fp8_logits(q, s, w, ws, out)

        same(*both(call))
    same(*both(lambda: pstat.fp8_quantize(x[:0])))


def test_beams(both):
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(6, 500, generator=g, device="cuda")
    s = torch.randn(2, 3, generator=g, device="cuda")
    same(*both(lambda: pstat.beam_select(z, s, 5)))
    cache = torch.randn(6, 2, 9, 4, generator=g, device="cuda")
    parents = torch.tensor([[1, 0, 2], [2, 2, -1]], device="cuda")
    parents_to = torch.tensor([[1, 0], [2, 2]], device="cuda")

    def call(out):
        x = cache.clone()
        states = [x[:, :, :5], x[:, :, 5:].transpose(1, 3), x[:, :, 6]]
        if out:
            count = states[0]._version
            got = pstat.beam_reorder(states[:2], parents, out=states[:2])
            assert all(a is b for a, b in zip(got, states)) and states[0]._version > count
            return [x]
        return pstat.beam_reorder(states, parents_to)

    same(*both(lambda: call(True)))
    same(*both(lambda: call(False)))


def test_refusals_and_devices(both):
    p = torch.zeros(10, device="cuda")
    m, v = pstat.adamw_state(p)

    def refused():
        try:
            pstat.beam_reorder([p], torch.zeros(1, 5, dtype=torch.int64, device="cuda"), out=[p])
        except (ValueError, pstat.PstatError) as e:
            return str(e)

    a, b = both(refused)
    assert a == b and a

    def calls():
        for f in (lambda: pstat.adamw_step(p, p, m, v, 1, 1e-3),
                  lambda: pstat.adamw_step(p, p.clone(), m, v, 0, 1e-3),
                  lambda: pstat.adamw_step(p, p[:5].clone(), m, v, 1, 1e-3),
                  lambda: pstat.beam_select(torch.zeros(65, 4, device="cuda"),
                                            torch.zeros(1, 65, device="cuda"), 2),
                  lambda: pstat.fp8_quantize(p.view(2, 5), 3)):
            with pytest.raises((ValueError, pstat.PstatError)) as e:
                f()
            yield str(e.value)

    a, b = both(lambda: list(calls()))
    assert a == b
