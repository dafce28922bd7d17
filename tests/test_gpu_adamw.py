"""The AdamW step against its formula.

Moments are products and sums that are each rounded once: fp32 moments have to equal
numpy's, 8-bit codes those that the oracle finds by search.  A parameter is, in units
of 2^-24: of itself, 1 for the decay's constant, 1 for its product and half for the
last sum (3 covers them); of the update lr m / (...), 4 each for the root and the
quotient (2^-22), 1 for each of size, root constant, and fused sums: below 16.  A bf16
parameter adds half a step of bf16, 2^-8, or a whole one where it is drawn."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import adamw as oadam

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HYPER = dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)


def _case(n, seed, p_type, g_type, bits, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def at(x, dtype):  # a tensor that starts `off` elements into its storage
        store = torch.empty(n + off, dtype=dtype, device="cuda")
        store[off:] = x
        return store[off:]

    wide = torch.exp(2 * torch.randn(n, generator=g, device="cuda"))
    p = at(torch.randn(n, generator=g, device="cuda"), p_type)
    grad = at(1e-3 * wide * torch.randn(n, generator=g, device="cuda"), g_type)
    m = 1e-3 * wide * torch.randn(n, generator=g, device="cuda")
    v = (1e-3 * wide * torch.rand(n, generator=g, device="cuda")).square()
    m[::7] = 0
    v[::11] = 0
    if bits == 8:
        def code(x, kind):
            return at_state(oadam.encode(x.cpu().numpy(), [1 << 19] * n, kind))

        def at_state(c):
            store = torch.empty(len(c) + off, dtype=torch.uint8, device="cuda")
            store[off:] = torch.from_numpy(c).cuda()
            return store[off:]

        m, v = code(m, "m"), code(v, "v")
    else:
        m, v = at(m, F32), at(v, F32)
    return p, grad, m, v


def _expect(p, g, m, v, bits, seed, index, step, lr, factor, betas, eps, weight_decay):
    n = p.numel()
    m0 = oadam.decode(m.cpu().numpy(), n, "m") if bits == 8 else m.cpu().numpy()
    v0 = oadam.decode(v.cpu().numpy(), n, "v") if bits == 8 else v.cpu().numpy()
    m1, v1 = oadam.moments(m0, v0, g.float().cpu().numpy(), factor, *betas)
    exact = oadam.parameter(p.double().cpu().numpy(), m1, v1, step, lr, *betas, eps, weight_decay)
    if bits == 8:
        to_m, to_v, _ = oadam.draws(seed, index, n)
        return exact, oadam.encode(m1, to_m, "m"), oadam.encode(v1, to_v, "v")
    return exact, m1, v1


def _check(p_new, p_old, m, v, want, bits, drawn):
    exact, wm, wv = want
    wm, wv = torch.from_numpy(np.asarray(wm)).cuda(), torch.from_numpy(np.asarray(wv)).cuda()
    if bits == 32:
        wm, wv = wm.view_as(m), wv.view_as(v)
        assert torch.equal(m.view(torch.int32), wm.view(torch.int32))
        assert torch.equal(v.view(torch.int32), wv.view(torch.int32))
    else:
        assert torch.equal(m, wm) and torch.equal(v, wv)
    exact = torch.from_numpy(exact).cuda()
    update = (exact - p_old.double()).abs()
    room = 2.0**-24 * (3 * p_old.double().abs() + 16 * update) + 2.0**-149
    if p_new.dtype == BF16:
        room = room * (1 + 2.0**-8) + (2.0**-7 if drawn else 2.0**-8) * exact.abs() + 2.0**-133
    bad = (p_new.double() - exact).abs() > room
    assert not bool(bad.any()), (int(bad.sum()), p_new[bad][:3], exact[bad][:3])


SIZES = [1, 3, 127, 128, 129, 1000, 4096, 4097, 12800]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type", list(itertools.product([F32, BF16], repeat=2)))
@pytest.mark.parametrize("seed", [None, 12345678901234567])
def test_list(cuda_lib, bits, p_type, g_type, seed):
    """One list of many sizes, aligned and not."""
    cases = [_case(n, 3 + i, p_type, g_type, bits, off) for i, (n, off) in
             enumerate([(n, 0) for n in SIZES] + [(1000, 1), (700, 3), (0, 0)])]
    ps, gs, ms, vs = (list(x) for x in zip(*cases))
    old = [p.clone() for p in ps]
    want = [_expect(p, g, m, v, bits, seed, i, 5, 1e-2, 1.0, **HYPER)
            for i, (p, g, m, v) in enumerate(cases)]
    got = cuda_lib.adamw_step(ps, gs, ms, vs, 5, 1e-2, **HYPER, seed=seed)
    assert all(a is b for a, b in zip(got, ps))
    for p, o, m, v, w in zip(ps, old, ms, vs, want):
        _check(p, o, m, v, w, bits, seed is not None)


def test_many_tensors_of_mixed_kinds(cuda_lib):
    """More tensors than one launch takes; a tensor's draws go by its place in the list."""
    kinds = list(itertools.product([F32, BF16], [F32, BF16], [32, 8]))
    cases = [_case(1 + i % 9, i, *kinds[i % 8]) for i in range(1300)]
    bits = [kinds[i % 8][2] for i in range(1300)]
    ps, gs, ms, vs = (list(x) for x in zip(*cases))
    old = [p.clone() for p in ps]
    want = [_expect(*c, b, 9, i, 1, 1e-3, 1.0, **HYPER) for i, (c, b) in enumerate(zip(cases, bits))]
    cuda_lib.adamw_step(ps, gs, ms, vs, 1, 1e-3, **HYPER, seed=9)
    for p, o, m, v, w, b in zip(ps, old, ms, vs, want, bits):
        _check(p, o, m, v, w, b, True)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_on_the_way(cuda_lib, bits):
    """The step with a norm is the step on the clipped fp32 gradients; one that is
    not finite changes nothing."""
    p, g, m, v = _case(5000, 1, F32, F32, bits)
    norm = cuda_lib.grad_norm([g])
    for limit in (0.25 * norm.item(), 4 * norm.item(), 0.0):
        limit = float(np.float32(limit))
        a = [x.clone() for x in (p, m, v)]
        factor = min(np.float32(1), np.float32(limit) / np.float32(norm.item()))
        want = _expect(a[0], g, a[1], a[2], bits, None, 0, 3, 1e-3, factor, **HYPER)
        cuda_lib.adamw_step(a[0], g, a[1], a[2], 3, 1e-3, **HYPER, norm=norm, max_norm=limit)
        _check(a[0], p, a[1], a[2], want, bits, False)
    for bad in (math.inf, math.nan):
        err = cuda_lib.new_error_flag("cuda:0")
        a = [x.clone() for x in (p, m, v)]
        cuda_lib.adamw_step(a[0], g, a[1], a[2], 3, 1e-3, **HYPER, max_norm=1.0,
                            norm=torch.tensor(bad, device="cuda"), dev_error=err)
        assert err.item() == cuda_lib.DEV_NONFINITE
        assert all(torch.equal(x, y) for x, y in zip(a, (p, m, v)))


def test_values_at_the_ends(cuda_lib):
    """Zeros, subnormals, the largest numbers, infinities and NaN in a block of codes."""
    n = 384
    g = torch.zeros(n, device="cuda")
    g[:8] = torch.tensor([0.0, 1e-45, 1e-30, 1e18, -1e18, math.inf, -math.inf, math.nan])
    g[128:136] = torch.tensor([1e-42, -1e-42, 1e-45, 3e-39, 0, 0, 1e-38, 1e-22])
    for seed in (None, 3):
        p = torch.ones(n, device="cuda")
        m, v = cuda_lib.adamw_state(p, 8)
        want = _expect(p, g, m, v, 8, seed, 0, 1, 1e-3, 1.0, **HYPER)
        cuda_lib.adamw_step([p], [g], [m], [v], 1, 1e-3, **HYPER, seed=seed)
        assert torch.equal(m.cpu(), torch.from_numpy(want[1]))
        assert torch.equal(v.cpu(), torch.from_numpy(want[2]))
        lost = torch.zeros(n, dtype=torch.bool, device="cuda")
        lost[5:8] = True
        assert torch.equal(torch.isnan(p), lost)
        (am,), (av,) = cuda_lib.adamw_moments([m], [v], [p])
        assert torch.equal(torch.isnan(am), lost) and torch.equal(torch.isnan(av), lost)
        assert np.array_equal(am.double().cpu().numpy(), oadam.decode(m.cpu().numpy(), n, "m"),
                              equal_nan=True)
        assert np.array_equal(av.double().cpu().numpy(), oadam.decode(v.cpu().numpy(), n, "v"),
                              equal_nan=True)


@pytest.mark.parametrize("off", [0, 1, 2])
def test_moments_of_a_list(cuda_lib, off):
    cases = [_case(n, n, F32, F32, 8, off) for n in (1, 128, 129, 5000)]
    ps, _, ms, vs = (list(x) for x in zip(*cases))
    outs = [[torch.full((p.numel() + off,), 7.0, device="cuda")[off:] for p in ps] for _ in range(2)]
    got = cuda_lib.adamw_moments(ms, vs, ps, out=outs)
    for kind, states, new in (("m", ms, got[0]), ("v", vs, got[1])):
        for p, s, x in zip(ps, states, new):
            assert np.array_equal(x.double().cpu().numpy(),
                                  oadam.decode(s.cpu().numpy(), p.numel(), kind))


def test_drawn_roundings_follow_the_mean(cuda_lib):
    """A gradient whose square lies 2% above v: rounded to nearest v stands still, drawn
    it follows (a random walk of 4096 elements and 200 steps of at most 2^-3 each way,
    whose mean is off by at most 4 sqrt(200 / 4096) / 16 < 0.06)."""
    n = 4096
    for seed, lo, hi in ((None, 0.99, 1.01), (1, 1.10, 1.25)):
        p = torch.zeros(n, device="cuda")
        g = torch.full((n,), math.sqrt(1.2), device="cuda")
        m, v = cuda_lib.adamw_state(p, 8)
        v[:n] = 30 * 8 + 0
        v[n:] = 127  # 1.0 everywhere
        for t in range(200):
            cuda_lib.adamw_step([p], [g], [m], [v], t + 1, 0.0, betas=(0.9, 0.98),
                                seed=None if seed is None else seed + t)
        mean = cuda_lib.adamw_moments([m], [v], [p])[1][0].double().mean().item()
        assert lo <= mean <= hi, (seed, mean)


def test_same_call_same_bits_and_other_seeds(cuda_lib):
    p, g, m, v = _case(20000, 4, BF16, BF16, 8)
    runs = []
    for seed in (1, 1, 2, 1 << 40, -1):
        a = [x.clone() for x in (p, m, v)]
        cuda_lib.adamw_step(a[0], g, a[1], a[2], 2, 1e-3, seed=seed)
        runs.append(a)
    assert all(torch.equal(x, y) for x, y in zip(runs[0], runs[1]))
    for i, j in itertools.combinations((0, 2, 3, 4), 2):
        assert not torch.equal(runs[i][1], runs[j][1])


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step(cuda_lib, bits):
    """Step, learning rate and seed read from the device at each replay."""
    p, g, m, v = _case(9000, 6, BF16, F32, bits)
    a, b = [x.clone() for x in (p, m, v)], [x.clone() for x in (p, m, v)]
    step = torch.ones((), dtype=torch.int64, device="cuda")
    lr = torch.full((), 1e-2, device="cuda")
    seed = torch.full((), 77, dtype=torch.int64, device="cuda")
    cuda_lib.adamw_step([p.clone()], [g], [m.clone()], [v.clone()], step, lr, seed=seed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.adamw_step(a[0], g, a[1], a[2], step, lr, seed=seed)
    for t in range(1, 5):
        rate = float(np.float32(1e-2 / t))
        lr.fill_(rate)
        step.fill_(t)
        seed.fill_(70 + t)
        graph.replay()
        cuda_lib.adamw_step(b[0], g, b[1], b[2], t, rate, seed=70 + t)
        torch.cuda.synchronize()
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        assert torch.equal(a[0], b[0])


def test_streams_and_counters(cuda_lib):
    p, g, m, v = _case(100000, 8, F32, F32, 32)
    a = [x.clone() for x in (p, m, v)]
    cuda_lib.adamw_step(a[0], g, a[1], a[2], 1, 1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    counts = [x._version for x in (p, m, v, g)]
    with torch.cuda.stream(side):
        cuda_lib.adamw_step(p, g, m, v, 1, 1e-3)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, (p, m, v)))
    assert [x._version - c for x, c in zip((p, m, v, g), counts)] == [1, 1, 1, 0]


def test_refusals(cuda_lib):
    p = torch.zeros(300, device="cuda")
    g = torch.zeros(300, device="cuda")
    m, v = cuda_lib.adamw_state(p)
    m8, v8 = cuda_lib.adamw_state(p, 8)
    assert m8.numel() == 303
    ok = dict(step=1, lr=1e-3)
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=math.nan), dict(betas=(1.0, 0.9)),
                dict(betas=(0.9, -0.1)), dict(eps=-1e-8), dict(weight_decay=math.inf)):
        with pytest.raises(cuda_lib.PstatError):
            cuda_lib.adamw_step(p, g, m, v, **{**ok, **bad})
    with pytest.raises(cuda_lib.PstatError):  # overlaps
        cuda_lib.adamw_step(p, p, m, v, **ok)
    with pytest.raises(cuda_lib.PstatError):
        cuda_lib.adamw_step([p, p], [g, g], [m, v], [torch.zeros_like(m), torch.zeros_like(m)], **ok)
    for args in ((p[:299], g, m, v), (p, g, m, v8), (p, g, m8, v), (p, g, m[:100], v[:100]),
                 (p, g.cpu(), m, v), ([], [], [], []), ([p], [g, g], [m], [v]), (p[::2], g[::2], m, v)):
        with pytest.raises(ValueError):
            cuda_lib.adamw_step(*args, **ok)
    with pytest.raises(TypeError):
        cuda_lib.adamw_step(p.half(), g, m, v, **ok)
    with pytest.raises(ValueError):
        cuda_lib.adamw_step(p, g, m, v, **ok, max_norm=1.0)
    with pytest.raises(ValueError):
        cuda_lib.adamw_step(p, g, m, v, torch.ones((), device="cuda"), 1e-3)
    with pytest.raises(ValueError):
        cuda_lib.adamw_moments([m], [v], [p])
    with pytest.raises(ValueError):
        cuda_lib.adamw_state(p, 4)
    assert not bool(p.any())


@pytest.mark.parametrize("p_type,g_type,seed", [(BF16, BF16, 7), (BF16, BF16, None), (F32, F32, 7), (BF16, F32, 7),
                                                (F32, BF16, None)])
def test_large_8_bit_tensors_in_any_place(cuda_lib, p_type, g_type, seed):
    """Tensors on 16 bytes take another way than those that are not: the same bits, also
    where blocks hold zeros, NaN, infinities and values far below their largest, and
    past 32 blocks for each warp of the GPU."""
    n = 13_000_077
    gen = torch.Generator(device="cuda").manual_seed(8)
    start = [torch.randn(n, generator=gen, device="cuda").to(p_type),
             (torch.randn(n, generator=gen, device="cuda") *
              torch.exp2(torch.randint(-40, 3, (n,), generator=gen, device="cuda").float())).to(g_type)]
    start[1][torch.randint(0, n, (20000,), generator=gen, device="cuda")] = 0
    start[1][100 * 128:110 * 128] = 0
    for value, count in ((math.nan, 30), (math.inf, 30)):
        start[1][torch.randint(0, n, (count,), generator=gen, device="cuda")] = value
        start[0][torch.randint(0, n, (count,), generator=gen, device="cuda")] = value
    results = []
    for off in (0, 1):
        p, g = (torch.empty(n + off, dtype=x.dtype, device="cuda")[off:].copy_(x) for x in start)
        m, v = (torch.zeros(n + -(-n // 128) + off, dtype=torch.uint8, device="cuda")[off:] for _ in range(2))
        for step in (1, 2, 3):
            cuda_lib.adamw_step(p, g, m, v, step, 1e-2, **HYPER, seed=None if seed is None else seed + step)
        results.append((p, m, v))
    (p, m, v), (q, mq, vq) = results
    assert torch.equal(m, mq) and torch.equal(v, vq)
    assert torch.equal(torch.isnan(p), torch.isnan(q))
    assert torch.equal(torch.nan_to_num(p, nan=0.5), torch.nan_to_num(q, nan=0.5))
    assert 50 < int(torch.isnan(p).sum()) < 1000
