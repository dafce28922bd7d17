"""The operators of a decoding step and of a training step one after another, as they are
used, eagerly and captured, and at sizes past 32 bits."""
import numpy as np
import pytest
import torch

from oracle import beams as obeams
from oracle import filters as oflt
from test_gpu_adamw import HYPER, _check, _expect

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ---- a beam search with an 8-bit head and a cache -----------------------------------

class Search:
    """A toy model: a beam's hidden state is the mean of what its cache holds, one vector of
    `d` numbers for each token so far."""

    def __init__(self, lib, B=3, beams=4, V=5003, d=256, steps=6, ld=8):
        g = torch.Generator(device="cuda").manual_seed(11)
        self.lib, self.B, self.beams, self.steps, self.d = lib, B, beams, steps, d
        self.emb = torch.randn(V, d, generator=g, device="cuda")
        W = torch.randn(V, d, generator=g, device="cuda").to(BF16)
        self.W, self.W_scale = lib.fp8_quantize(W, 128)
        self.start = torch.randint(0, V, (B,), generator=g, device="cuda").repeat_interleave(beams)
        self.cache = torch.empty(B * beams, 2, steps + ld, d // 2, device="cuda")
        self.history = torch.empty(B * beams, steps, dtype=torch.int64, device="cuda")
        self.scores = torch.empty(B, beams, device="cuda")
        self.parent = torch.empty(B, beams, dtype=torch.int64, device="cuda")
        self.token = torch.empty(B, beams, dtype=torch.int64, device="cuda")
        self.at = torch.empty(1, dtype=torch.int64, device="cuda")
        self.err = lib.new_error_flag("cuda:0")
        self.reset()

    def reset(self):
        self.cache.zero_()
        self.history.fill_(-1)
        self.at.zero_()
        self.scores.fill_(-float("inf"))  # the beams of a search are alike at first:
        self.scores[:, 0] = 0             # one of them goes on
        self.remember(self.start)

    def remember(self, token):
        self.cache.index_copy_(2, self.at, self.emb[token].view(len(token), 2, 1, self.d // 2))

    def logits(self):
        hidden = (self.cache[:, :, :self.steps].sum(2) / (self.at + 1)).reshape(-1, self.d).to(BF16)
        q, scale = self.lib.fp8_quantize(hidden, dev_error=self.err)
        return self.lib.fp8_logits(q, scale, self.W, self.W_scale, dev_error=self.err)

    def step(self):
        z = self.logits()
        self.lib.beam_select(z, self.scores, self.beams, out=(self.scores, self.parent, self.token),
                             dev_error=self.err)
        states = [self.cache[:, :, :self.steps], self.history]
        self.lib.beam_reorder(states, self.parent, out=states, dev_error=self.err)
        token = self.token.view(-1)
        self.history.index_copy_(1, self.at, token.view(-1, 1))
        self.at += 1
        self.remember(token)
        return z


def test_beam_search(cuda_lib):
    s = Search(cuda_lib)
    B, beams = s.B, s.beams
    for i in range(s.steps):
        before = [x.clone() for x in (s.scores, s.cache, s.history)]
        z = s.step()
        want = obeams.select(z.double().cpu().numpy().reshape(B, beams, -1), before[0].cpu().numpy(), beams)
        assert np.array_equal(s.parent.cpu().numpy(), want[1])
        assert np.array_equal(s.token.cpu().numpy(), want[2])
        assert (np.abs(s.scores.cpu().numpy() - want[0]) <= 6e-6 + 2.0**-24 * np.abs(want[0])).all()
        row = (s.parent + beams * torch.arange(B, device="cuda")[:, None]).view(-1)
        assert torch.equal(s.cache[:, :, :i + 1], before[1][row][:, :, :i + 1])
        assert torch.equal(s.history[:, :i], before[2][row][:, :i])
    assert s.err.item() == 0
    # Each beam's score is the sum of the log-probabilities of its tokens, taken one by one:
    # per step 1e-5 for the log-probability and 6e-6 + 2^-24 |score| for the search's.
    scores, history = s.scores.clone(), s.history.clone()
    assert len({tuple(x) for x in history.tolist()}) == B * beams
    s.reset()
    total = torch.zeros(B * beams, dtype=torch.float64, device="cuda")
    for i in range(s.steps):
        total += cuda_lib.forward(s.logits(), history[:, i])[0].double()
        s.at += 1
        s.remember(history[:, i])
    room = s.steps * (1.6e-5 + 2.0**-24 * float(total.abs().max()))
    assert float((total - scores.view(-1).double()).abs().max()) <= room


def test_captured_beam_search(cuda_lib):
    s = Search(cuda_lib)
    for _ in range(s.steps):
        s.step()
    want = [x.clone() for x in (s.scores, s.history, s.cache)]
    s.reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(2):
        s.reset()
        for _ in range(s.steps):
            graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (s.scores, s.history, s.cache)))


def test_sampling_from_an_8_bit_head(cuda_lib):
    s = Search(cuda_lib, B=5, beams=1)
    u = torch.rand(5, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    z = s.logits()
    token, logprob = cuda_lib.sample(z, u, 0.9, 50, 0.95)
    for i in range(5):
        v, lp, near = oflt.sample(z[i].double().cpu().numpy(), u[i].item(), float(np.float32(0.9)), 50,
                                  float(np.float32(0.95)))
        assert near < 1e-12 or (token[i].item() == v and abs(logprob[i].item() - lp) <= 1e-5)


def test_searches_on_two_streams_at_once(cuda_lib):
    a, b = Search(cuda_lib), Search(cuda_lib, B=2, beams=7, V=20001)
    want = []
    for s in (a, b):
        for _ in range(s.steps):
            s.step()
        want.append([x.clone() for x in (s.scores, s.history)])
        s.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(a.steps):
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                s.step()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert torch.equal(s.scores, w[0]) and torch.equal(s.history, w[1])


# ---- a training step -------------------------------------------------------------------

class Training:
    """A head and a vector, by the head's policy gradient, the clipped AdamW step and the
    head's codes for decoding."""

    def __init__(self, lib, bits, T=96, V=500, d=256):
        g = torch.Generator(device="cuda").manual_seed(12)
        self.lib = lib
        self.hidden = torch.randn(T, d, generator=g, device="cuda").to(BF16)
        self.y = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.y[5] = -100
        self.w = -torch.rand(T, generator=g, device="cuda")
        self.params = [(0.1 * torch.randn(V, d, generator=g, device="cuda")).to(BF16),
                       torch.randn(77, generator=g, device="cuda")]
        self.grads = [torch.zeros(V, d, device="cuda"), torch.randn(77, generator=g, device="cuda")]
        self.dh = torch.zeros(T, d, device="cuda")
        self.m, self.v = (list(x) for x in zip(*(lib.adamw_state(p, bits) for p in self.params)))
        self.t = torch.ones(1, dtype=torch.int64, device="cuda")
        self.lr = torch.full((1,), 1e-2, device="cuda")
        self.norm = torch.empty((), device="cuda")
        self.codes = lib.fp8_quantize(self.params[0], 128)
        self.err = lib.new_error_flag("cuda:0")

    def state(self):
        return [x.view(torch.uint8) for x in (*self.params, *self.m, *self.v, *self.codes, self.norm.view(1))]

    def step(self):
        lib = self.lib
        lp, ent, rs = lib.lmhead_forward(self.hidden, self.params[0], self.y, dev_error=self.err)
        self.grads[0].zero_()
        lib.lmhead_backward(self.hidden, self.params[0], self.y, self.w, rs, dhidden=self.dh, dW=self.grads[0],
                            dev_error=self.err)
        lib.grad_norm(self.grads, out=self.norm, dev_error=self.err)
        lib.adamw_step(self.params, self.grads, self.m, self.v, self.t, self.lr, **HYPER, norm=self.norm,
                       max_norm=0.5, seed=self.t, dev_error=self.err)
        lib.fp8_quantize(self.params[0], 128, out=self.codes, dev_error=self.err)
        self.t += 1


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step(cuda_lib, bits):
    s = Training(cuda_lib, bits)
    for step in (1, 2):
        old = [x.clone() for x in s.params]
        ms, vs = [x.clone() for x in s.m], [x.clone() for x in s.v]
        s.step()
        factor = min(np.float32(1), np.float32(0.5) / s.norm.cpu().numpy())
        assert factor < 1 and s.err.item() == 0
        for i, p in enumerate(s.params):
            want = _expect(*(x.view(-1) for x in (old[i], s.grads[i], ms[i], vs[i])), bits, step, i, step,
                           float(s.lr), factor, **HYPER)
            _check(p.view(-1), old[i].view(-1), s.m[i].view(-1), s.v[i].view(-1), want, bits, p.dtype == BF16)
        q, scale = cuda_lib.fp8_quantize(s.params[0], 128)
        assert torch.equal(q.view(torch.uint8), s.codes[0].view(torch.uint8))
        assert torch.equal(scale, s.codes[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training_step(cuda_lib, bits):
    eager, s = Training(cuda_lib, bits), Training(cuda_lib, bits)
    first = [x.clone() for x in s.state()]
    for _ in range(3):
        eager.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    assert all(torch.equal(a, b) for a, b in zip(first[:-1], s.state()))  # nothing has run yet
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(eager.state(), s.state()))
    assert s.t.item() == 4 and s.err.item() == 0


# ---- past 32 bits ------------------------------------------------------------------------

def test_adamw_past_32_bits_of_elements(cuda_lib):
    """The last 1024 elements, from 2^32 on, are as the first 1024: alike to nearest, drawn
    apart from them."""
    n = (1 << 32) + 1024
    g = torch.zeros(n, dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(13)
    part = torch.randn(1024, generator=gen, device="cuda").to(BF16)
    g[:1024] = part
    g[n - 1024:] = part
    for seed in (None, 5):
        p = torch.ones(n, dtype=BF16, device="cuda")
        m, v = cuda_lib.adamw_state(p, 8)
        cuda_lib.adamw_step(p, g, m, v, 1, 1e-2, **HYPER, seed=seed)
        blocks = n // 128
        heads = [torch.cat([x[:1024], x[n:n + 8]]) for x in (m, v)]
        tails = [torch.cat([x[n - 1024:n], x[n + blocks - 8:]]) for x in (m, v)]
        zero = torch.zeros(1032, dtype=torch.uint8, device="cuda")
        want = _expect(torch.ones(1024, device="cuda"), part, zero, zero, 8, seed, 0, 1, 1e-2, 1.0, **HYPER)
        _check(p[:1024], torch.ones(1024, device="cuda"), *heads, want, 8, seed is not None)
        assert not bool(m[1024:n - 1024].any()) and not bool(v[1024:n - 1024].any())
        if seed is None:
            assert torch.equal(p[:1024], p[n - 1024:])
            assert all(torch.equal(a, b) for a, b in zip(heads, tails))
        else:
            assert not torch.equal(heads[0][:1024], tails[0][:1024])
            assert all(torch.equal(a[1024:], b[1024:]) for a, b in zip(heads, tails))
        del p, m, v


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_past_32_bits_of_elements(cuda_lib, rows):
    T, K = 131200, 32768  # 2^32 + 4.2 million elements
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(14)
    x[-128:] = torch.randn(128, K, generator=gen, device="cuda").to(BF16)
    q, s = cuda_lib.fp8_quantize(x, rows)
    want_q, want_s = cuda_lib.fp8_quantize(x[-128:], rows)
    assert torch.equal(q[-128:].view(torch.uint8), want_q.view(torch.uint8))
    assert torch.equal(s[-want_s.shape[0]:], want_s)
    assert not bool(q[:-128].view(torch.uint8).any()) and bool((s[:-want_s.shape[0]] == 1).all())


@pytest.mark.parametrize("out", [BF16, F32])
def test_logits_past_32_bits_of_elements(cuda_lib, out):
    T, V, K = 28300, 151936, 144  # 4.3 billion logits
    gen = torch.Generator(device="cuda").manual_seed(15)
    q, s = cuda_lib.fp8_quantize(torch.randn(T, K, generator=gen, device="cuda"))
    W, Ws = cuda_lib.fp8_quantize(torch.randn(V, K, generator=gen, device="cuda"), 128)
    got = cuda_lib.fp8_logits(q, s, W, Ws, out)
    for at in (slice(0, 3), slice(14130, 14140), slice(T - 130, T)):
        assert torch.equal(got[at], cuda_lib.fp8_logits(q[at], s[at], W, Ws, out))


def test_beams_past_32_bits_of_elements(cuda_lib):
    B, beams, V = 450, 64, 151936  # 4.4 billion logits
    gen = torch.Generator(device="cuda").manual_seed(16)
    z = torch.zeros(B * beams, V, dtype=BF16, device="cuda")
    z[-64:] = torch.randn(64, V, generator=gen, device="cuda").to(BF16)
    scores = -torch.rand(B, beams, generator=gen, device="cuda")
    got = cuda_lib.beam_select(z, scores, 16)
    want = cuda_lib.beam_select(z[-64:], scores[-1:], 16)
    assert all(torch.equal(a[-1:], b) for a, b in zip(got, want))
    # all logits equal: the best beam's first tokens
    best = scores.argmax(1)
    assert torch.equal(got[1][:-1], best[:-1, None].expand(-1, 16))
    assert torch.equal(got[2][:-1], torch.arange(16, device="cuda").expand(B - 1, 16))


# ---- calls that the tests of each operator do not make --------------------------------------

def test_scores_in_place_and_overlaps(cuda_lib):
    gen = torch.Generator(device="cuda").manual_seed(17)
    z = torch.randn(30, 3001, generator=gen, device="cuda")
    z[10:20] = z[:10]  # near ties, whose sums are taken anew
    scores = -torch.rand(3, 10, generator=gen, device="cuda")
    want = cuda_lib.beam_select(z, scores, 10)
    parent, token = torch.empty_like(want[1]), torch.empty_like(want[2])
    got = scores.clone()
    cuda_lib.beam_select(z, got, 10, out=(got, parent, token))
    assert all(torch.equal(a, b) for a, b in zip(want, (got, parent, token)))
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_select(z, scores, 10, out=(got, parent, parent))
    with pytest.raises(cuda_lib.PstatError):  # rows of 5 over rows of 10
        cuda_lib.beam_select(z, scores, 5, out=(scores.view(-1)[:15].view(3, 5), parent.view(-1)[:15].view(3, 5),
                                                token.view(-1)[:15].view(3, 5)))
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_select(z, scores, 10, out=(z.view(-1)[:30].view(3, 10), parent, token))
    parents = torch.zeros(3, 10, dtype=torch.int64, device="cuda")
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.beam_reorder([parents.view(30, 1)], parents, out=[parents.view(30, 1)])
    x = torch.zeros(64, 128, device="cuda")
    buffer = x.view(torch.float8_e4m3fn).view(-1)
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.fp8_quantize(x, out=(buffer[:64 * 128].view(64, 128), torch.empty(64, 1, device="cuda")))
    q, s = cuda_lib.fp8_quantize(x)
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.fp8_logits(q, s, q, torch.ones(1, 1, device="cuda"),
                            out=q.view(BF16).view(64, 64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("beams,V,n", [(3, 10007, 32), (3, 10007, 1), (1, 2000, 31), (2, 30000, 32)])
def test_few_values_in_few_maxima(cuda_lib, dtype, beams, V, n):
    """Most logits at the maximum: far more candidates than a round of sorting takes."""
    gen = torch.Generator(device="cuda").manual_seed(V + n)
    z = torch.randint(0, 2, (2 * beams, V), generator=gen, device="cuda").to(dtype)
    z[:beams] = 1  # all of them
    scores = torch.zeros(2, beams, device="cuda")
    got = cuda_lib.beam_select(z, scores, n)
    want = obeams.select(z.double().cpu().numpy().reshape(2, beams, V), scores.cpu().numpy(), n)
    # Beams whose rows have equal sums tie exactly; others are told apart by their sums.
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])


def test_padded_batch_and_empty_calls(cuda_lib):
    """Searches that are over (no beam goes on) beside others, and calls with no rows."""
    gen = torch.Generator(device="cuda").manual_seed(18)
    z = torch.randn(12, 500, generator=gen, device="cuda")
    z[4:8] = float("nan")  # of no consequence without a score
    scores = -torch.rand(3, 4, generator=gen, device="cuda")
    scores[1] = -float("inf")
    err = cuda_lib.new_error_flag("cuda:0")
    score, parent, token = cuda_lib.beam_select(z, scores, 8, dev_error=err)
    assert err.item() == 0
    assert bool((score[1] == -float("inf")).all()) and bool((parent[1] == -1).all()) and bool((token[1] == -1).all())
    alone = cuda_lib.beam_select(z[8:], scores[2:], 8)
    assert all(torch.equal(a[2:], b) for a, b in zip((score, parent, token), alone))
    state = torch.randn(12, 40, generator=gen, device="cuda")
    want = state.clone()
    row = parent[:, :4] + 4 * torch.arange(3, device="cuda")[:, None]
    for b in (0, 2):
        want[4 * b:4 * b + 4] = state[row[b]]
    cuda_lib.beam_reorder([state], parent[:, :4].contiguous(), out=[state])
    assert torch.equal(state, want)  # the finished search's rows stay
    empty = cuda_lib.beam_select(z[:0], scores[:0], 3)
    assert [tuple(x.shape) for x in empty] == [(0, 3)] * 3
    assert cuda_lib.fp8_quantize(z[:0])[0].shape == (0, 500)
    x = torch.zeros(0, device="cuda")
    cuda_lib.adamw_step([x], [x], [x], [torch.zeros(0, device="cuda")], 1, 1e-3)


def test_zero_gradients_decay_only(cuda_lib):
    """Fresh moments under gradients of zero stay zero, and the parameter decays: its
    product's rounding and the constant's, 2^-23 of it."""
    for bits, eps in ((32, 1e-8), (8, 1e-8), (8, 1e-30)):
        p = torch.randn(1000, generator=torch.Generator(device="cuda").manual_seed(19), device="cuda")
        old, g = p.clone(), torch.zeros(1000, device="cuda")
        m, v = cuda_lib.adamw_state(p, bits)
        cuda_lib.adamw_step(p, g, m, v, 1, 0.5, eps=eps, weight_decay=0.25, seed=3 if bits == 8 else None)
        assert not bool(m.any()) and not bool(v.any())
        assert bool(((p.double() - 0.875 * old.double()).abs() <= 2.0**-23 * old.double().abs()).all())
