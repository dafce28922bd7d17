"""Sampling and the policy statistics under temperature and truncation,
against the float64 oracle (oracle/filters.py).

Tolerances.  Tokens and cuts are decisions of exact arithmetic and have to be
equal; a draw whose target lies within 1e-12 of a border of the cumulative
mass is skipped (the oracle's own float64 sums are no better than that).
logprob = x - ln S and entropy = ln S - U/S in fp32: each of x, ln S and U/S is
rounded a few times, so 8 half-steps of 2^-24 of the largest term's size
(|x| + |ln S| + |H|), and U is a sum of V fp32 terms whose error is bounded by
the forward statistics' own tolerance (helpers.TOL_FWD).
dlogits: p carries the error of x log2(e), |x| 2^-24 relative times a few, plus
the rounding to the output type: per element the rules of
helpers.assert_grad_close, 1e-3 relative for fp32 and one bf16 step for bf16.
Its Frobenius bound of 2.5e-3 holds for gradients of many entries of like size;
a truncated row can hang on one entry, which correct rounding alone moves by up
to half a step, 2^-8 = 3.9e-3 of its value.  So 2^-8 + 1e-4 is the bound here.
The label's own element, (w/t)(1 - p), inherits the absolute error of ln S: p
changes by p d(ln S).  A row without filters has ln S from fp32 sums, which near
S = 1 lie 2^-23 apart, off by half of that in each of the chunk's sum, the fold
and the logarithm: 4 x 2^-23 (w/t) is added there.
Exponentials and products below the least normal number, 2^-126, are flushed to
0: an element (w/t) e/S with S >= 1 may be off by 2^-126 (w/t) for the one and
2^-126 for the other.
"""
import math

import numpy as np
import pytest
import torch

from helpers import TOL_FWD, bf16_round, bf16_ulp, to_oracle
from oracle import filters as oflt

pytestmark = pytest.mark.gpu
IGN = -100
BF16, F32 = torch.bfloat16, torch.float32


def _rows(T, V, dtype, seed, pad=0, std=2.0, peak=0.0, mask=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = std * torch.randn(T, V, generator=g, device="cuda")
    if peak:
        n = min(V, 24)
        cols = torch.randint(0, V, (T, n), generator=g, device="cuda")
        z.scatter_add_(1, cols, peak * torch.rand(T, n, generator=g, device="cuda"))
    if mask:
        off = torch.rand(T, V, generator=g, device="cuda") < mask
        off[:, 0] = False
        z[off] = -math.inf
    store = torch.full((T, V + pad), 7.0, device="cuda", dtype=dtype)
    store[:, :V] = z.to(dtype)
    return store[:, :V], g


def _grad_close(g, b, room, what):
    """`room` [T, V]: what the label's element may be off besides."""
    a = g.double().cpu().numpy()
    if g.dtype == F32:
        ok = np.abs(a - b) <= 1e-3 * np.abs(b) + 1e-12 + room
    else:
        ok = np.abs(a - bf16_round(b)) <= np.maximum(1e-3 * np.abs(b), bf16_ulp(b)) + room
        assert np.linalg.norm(a - b) <= ((2.0**-8 + 1e-4) * np.linalg.norm(b)
                                         + np.linalg.norm(room)), what
    assert ok.all(), (what, np.argwhere(~ok)[0])


def _at(x, i):
    return x[i].item() if isinstance(x, torch.Tensor) else x


def _check_sample(lib, z, u, t=1.0, k=0, p=1.0, m=0.0, what=""):
    err = lib.new_error_flag(z.device)
    tok, lp = lib.sample(z, u, t, k, p, m, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0, err.item()
    zo = to_oracle(z)
    for i in range(z.shape[0]):
        v, want, near = oflt.sample(oflt.to_double(zo[i]), u[i].item(), _at(t, i), _at(k, i),
                                    _at(p, i), _at(m, i))
        if near < 1e-12:
            continue
        assert tok[i].item() == v, (what, i, tok[i].item(), v, near)
        x = abs(want) + 20
        assert abs(lp[i].item() - want) <= 8 * x * 2.0**-24, (what, i, lp[i].item(), want)
    return tok, lp


def _check_train(lib, z, y, w, t=1.0, k=0, p=1.0, m=0.0, out_dtype=None, what=""):
    err = lib.new_error_flag(z.device)
    lp, ent, rs, tau, idx = lib.filtered_forward(z, y, t, k, p, m, IGN, dev_error=err)
    g = lib.filtered_backward(z, y, w, rs, tau, idx, t, IGN, out_dtype, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0, err.item()
    zo = to_oracle(z)
    grads = []
    room = np.zeros(z.shape)
    tol = TOL_FWD[z.dtype]
    for i in range(z.shape[0]):
        zi = oflt.to_double(zo[i])
        a = (_at(t, i), _at(k, i), _at(p, i), _at(m, i))
        ref = oflt.forward(zi, int(y[i]), *a, IGN)
        assert idx[i].item() == ref["cut_index"], (what, i, idx[i].item(), ref)
        assert tau[i].item() == ref["cut_logit"], (what, i, tau[i].item(), ref)
        assert rs[i, 0].item() == ref["M"]
        big = abs(ref["lnS"]) + abs(ref["entropy"])
        assert abs(rs[i, 1].item() - ref["lnS"]) <= tol + 8 * big * 2.0**-24, (what, i)
        assert abs(ent[i].item() - ref["entropy"]) <= tol + 8 * big * 2.0**-24, (
            what, i, ent[i].item(), ref["entropy"])
        if math.isinf(ref["logprob"]):
            assert lp[i].item() == -math.inf, (what, i)
        else:
            big += abs(ref["logprob"])
            assert abs(lp[i].item() - ref["logprob"]) <= tol + 8 * big * 2.0**-24, (what, i)
        grads.append(oflt.backward(zi, int(y[i]), w[i].item(), *a, IGN))
        # below 2^-126 a weight and its product with w/t are taken as 0
        room[i] = 2.0**-126 * (1 + abs(w[i].item()) / _at(t, i))
        if y[i] != IGN:
            room[i, int(y[i])] += 4 * 2.0**-23 * abs(w[i].item()) / _at(t, i)
    _grad_close(g, np.stack(grads), room, what)
    return lp, ent, rs, tau, idx, g


def _labels(T, V, g):
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::5] = IGN
    w = torch.randn(T, generator=g, device="cuda")
    w[1::7] = 0.0
    return y, w


SETTINGS = [
    dict(),
    dict(t=0.7),
    dict(k=1),
    dict(k=50, t=0.8, p=0.95),
    dict(p=0.9),
    dict(p=0.3, t=1.7),
    dict(m=0.05, t=1.2),
    dict(k=200, p=0.99, m=0.01, t=0.5),
    dict(k=10**6),
    dict(p=1e-6),
    dict(m=1.0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 20011])
def test_sample_sizes(cuda_lib, dtype, V):
    z, g = _rows(9, V, dtype, V, pad=V % 3, peak=6.0)
    for n, s in enumerate(SETTINGS):
        u = torch.rand(9, generator=g, device="cuda")
        u[0] = 0.0
        u[1] = 1.0 - 2.0**-24
        _check_sample(cuda_lib, z, u, **s, what=f"V={V} {s}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("flat", [False, True])
def test_sample_wide(cuda_lib, dtype, flat):
    z, g = _rows(12, 151936, dtype, 5, peak=0.0 if flat else 18.0)
    for s in SETTINGS + [dict(k=5000), dict(k=100000, t=0.3), dict(p=0.999)]:
        _check_sample(cuda_lib, z, torch.rand(12, generator=g, device="cuda"), **s, what=str(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 2, 33, 1000, 20011])
def test_statistics_and_gradient(cuda_lib, dtype, V):
    z, g = _rows(11, V, dtype, V + 1, pad=V % 5, peak=6.0)
    y, w = _labels(11, V, g)
    for s in SETTINGS:
        _check_train(cuda_lib, z, y, w, **s, what=f"V={V} {s}")


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F32, F32), (F32, BF16)])
def test_statistics_wide(cuda_lib, dtype, out_dtype):
    z, g = _rows(6, 151936, dtype, 9, peak=16.0)
    y, w = _labels(6, 151936, g)
    y[1] = z[1].float().argmax()
    w[1] = 1.5
    for s in [dict(t=0.8, p=0.95), dict(k=40), dict(m=0.02, t=1.1), dict(t=1.3), dict(k=30000)]:
        _check_train(cuda_lib, z, y, w, **s, out_dtype=out_dtype, what=str(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties(cuda_lib, dtype):
    """Equal logits: constant rows, two-valued rows, +-0, more equal values
    than are sorted at once; the cut and the draw split them by index."""
    V = 30000
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.zeros(8, V, device="cuda", dtype=dtype)
    z[1, ::2] = -0.0
    z[2, ::3] = 1.0
    z[3] = torch.randint(0, 3, (V,), generator=g, device="cuda").to(dtype)
    z[4] = -3.0
    z[4, 17] = 2.0
    z[5, :100] = -math.inf
    z[6] = torch.randint(-2, 2, (V,), generator=g, device="cuda").to(dtype) * 40
    z[7] = -math.inf
    z[7, 5] = 1.0
    z[7, 9] = 1.0
    y, w = _labels(8, V, g)
    y[7], w[7] = 9, 1.0
    u = torch.tensor([0.0, 0.5, 0.25, 0.75, 0.9, 0.125, 1 - 2.0**-24, 0.5], device="cuda")
    for s in [dict(), dict(k=3), dict(k=20000), dict(p=0.5), dict(p=0.9, k=17000), dict(m=0.3),
              dict(p=0.25), dict(k=29950)]:
        _check_train(cuda_lib, z, y, w, **s, what=f"ties {s}")
        # constant rows put u S exactly on borders: the rule (first mass above
        # the target) is checked in whole numbers
        tok, _ = cuda_lib.sample(z, u, s.get("t", 1.0), s.get("k", 0), s.get("p", 1.0),
                                 s.get("m", 0.0))
        for i in range(8):
            kept, _, _, _, e = oflt.kept_set(oflt.to_double(to_oracle(z[i])), 1.0, s.get("k", 0),
                                             s.get("p", 1.0), s.get("m", 0.0))
            acc = np.cumsum(np.where(kept, e, 0.0))
            want = int(np.searchsorted(acc, u[i].item() * acc[-1], side="right"))
            near = np.min(np.abs(acc - u[i].item() * acc[-1])) / acc[-1]
            whole = np.all((e == 0) | (e == 1) | ~kept)
            if whole or near > 1e-12:
                assert tok[i].item() == want, (s, i, tok[i].item(), want)


def test_greedy(cuda_lib):
    z, g = _rows(7, 5003, BF16, 3)
    z[2, 4000] = z[2].max()
    z[3] = 1.0
    u = torch.rand(7, generator=g, device="cuda")
    tok, lp = cuda_lib.sample(z, u, 0.0)
    zf = z.float()
    want = torch.stack([(r == r.max()).nonzero()[0, 0] for r in zf])
    assert torch.equal(tok, want) and bool((lp == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_settings_per_row(cuda_lib, dtype):
    T, V = 40, 6007
    z, g = _rows(T, V, dtype, 8, pad=9, peak=8.0, mask=0.3)

    def pick(values, dt):
        return torch.tensor(values, device="cuda", dtype=dt)[
            torch.randint(0, len(values), (T,), generator=g, device="cuda")]

    t = pick([0.5, 0.9, 1.0, 1.4], torch.float32)
    k = pick([0, -1, 1, 30, 9000], torch.int32)
    p = pick([1.0, 0.9, 0.5], torch.float32)
    m = pick([0.0, 0.1], torch.float32)
    _check_sample(cuda_lib, z, torch.rand(T, generator=g, device="cuda"), t, k, p, m)
    y, w = _labels(T, V, g)
    _check_train(cuda_lib, z, y, w, t, k, p, m)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_values(cuda_lib, dtype):
    """Logits of the type's size, tiny differences, the temperature's limits."""
    V = 3001
    g = torch.Generator(device="cuda").manual_seed(6)
    big = torch.finfo(dtype).max
    z = torch.randn(6, V, generator=g, device="cuda")
    z[0] *= 1e30
    z[1, ::7] = -big
    z[2] = 1000.0 + z[2] * 1e-3
    z[3] *= 1e-20
    z[4, 3] = big
    z[5] *= 1e-6
    z = z.to(dtype)
    u = torch.rand(6, generator=g, device="cuda")
    y, w = _labels(6, V, g)
    for s in [dict(), dict(t=2.0**-20), dict(t=2.0**20), dict(p=0.9), dict(k=20, p=0.7),
              dict(t=1e-3, m=0.5), dict(t=1e4, m=0.9999)]:
        _check_sample(cuda_lib, z, u, **s, what=str(s))
        if s.get("t", 1.0) >= 1e-3:
            _check_train(cuda_lib, z, y, w, **s, what=str(s))


def test_undefined_rows_and_bad_values(cuda_lib):
    V = 500
    z, g = _rows(8, V, F32, 2)
    z[1] = -math.inf
    z[2, 7] = math.nan
    z[3, 9] = math.inf
    z[4, 11] = -math.nan
    u = torch.full((8,), 0.5, device="cuda")
    y = torch.zeros(8, dtype=torch.int64, device="cuda")
    y[5] = V
    err = cuda_lib.new_error_flag(z.device)
    tok, lp = cuda_lib.sample(z, u, top_p=0.9, dev_error=err)
    assert err.item() == cuda_lib.DEV_EMPTY_ROW
    assert tok[1:5].tolist() == [-1] * 4 and bool(lp[1:5].isnan().all())
    _check_sample(cuda_lib, z[5:], u[5:], p=0.9)
    err.zero_()
    lp, ent, rs, tau, idx = cuda_lib.filtered_forward(z, y, top_p=0.9, dev_error=err)
    assert err.item() == cuda_lib.DEV_EMPTY_ROW | cuda_lib.DEV_BAD_LABEL
    assert bool(lp[1:6].isnan().all()) and bool(ent[1:6].isnan().all())
    assert idx[1:5].tolist() == [-1] * 4 and bool(tau[1:5].isnan().all())
    err.zero_()
    gr = cuda_lib.filtered_backward(z, y, None, rs, tau, idx, dev_error=err)
    assert err.item() == cuda_lib.DEV_EMPTY_ROW | cuda_lib.DEV_BAD_LABEL
    assert bool(gr[1:6].isnan().all()) and not bool(gr[0].isnan().any())
    # values out of range, row by row
    ok = torch.randn(6, V, device="cuda")
    t = torch.tensor([1.0, -1.0, math.nan, 1.0, 1.0, 2.0**21], device="cuda")
    p = torch.tensor([1.0, 1.0, 1.0, 0.0, 1.0, 1.0], device="cuda")
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, 1.5, 0.0], device="cuda")
    err.zero_()
    tok, lp = cuda_lib.sample(ok, u[:6], t, 0, p, m, dev_error=err)
    assert err.item() == cuda_lib.DEV_BAD_PARAM
    assert tok[1:].tolist() == [-1] * 5 and 0 <= tok[0].item() < V
    err.zero_()
    bad_u = torch.tensor([0.5, 1.0, -0.1, math.nan, 0.2, 0.3], device="cuda")
    tok, lp = cuda_lib.sample(ok, bad_u, dev_error=err)
    assert err.item() == cuda_lib.DEV_BAD_PARAM and tok[1:4].tolist() == [-1] * 3
    err.zero_()
    lp, *_ = cuda_lib.filtered_forward(ok, y[:6] * 0, torch.zeros(6, device="cuda"), dev_error=err)
    assert err.item() == cuda_lib.DEV_BAD_PARAM and bool(lp.isnan().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batch_invariance(cuda_lib, dtype):
    """A row gives the same bits alone, in a small batch and in a large one, at
    any alignment and from call to call."""
    V, T = 30011, 700  # more rows than are resident at once: the other finish kernel
    z, g = _rows(T, V, dtype, 12, peak=12.0)
    z[::9] = _rows(len(z[::9]), V, dtype, 13)[0]  # flat rows, for the exact path
    u = torch.rand(T, generator=g, device="cuda")
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    for s in [(0.9, 0, 1.0, 0.0), (0.9, 0, 0.9, 0.0), (1.0, 40, 1.0, 0.0), (1.0, 0, 1.0, 0.05),
              (1.0, 4000, 0.99, 0.0)]:
        tok, lp = cuda_lib.sample(z, u, *s)
        full = cuda_lib.filtered_forward(z, y, *s)
        for a, b in ((0, 1), (7, 60), (250, 300), (600, 700)):
            store = torch.zeros(b - a, V + 5, dtype=dtype, device="cuda")
            store[:, 3:3 + V] = z[a:b]
            for part in (z[a:b], store[:, 3:3 + V]):
                tok2, lp2 = cuda_lib.sample(part, u[a:b], *s)
                assert torch.equal(tok2, tok[a:b])
                assert torch.equal(lp2.view(torch.int32), lp[a:b].view(torch.int32))
                for x, x2 in zip(full, cuda_lib.filtered_forward(part, y[a:b], *s)):
                    x, x2 = x[a:b].contiguous(), x2.contiguous()
                    if x.dtype == torch.float32:
                        x, x2 = x.view(torch.int32), x2.view(torch.int32)
                    assert torch.equal(x, x2), s


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_largest_vocabulary(cuda_lib, dtype):
    """2^20 columns: flat rows (bins with more logits than a list takes, nuclei of
    hundreds of thousands), ties, and a peaked row."""
    V = 1 << 20
    z, g = _rows(5, V, dtype, 17)
    z[1] *= 0.01
    z[2] = torch.randint(0, 40, (V,), generator=g, device="cuda").to(dtype) * 0.25
    z[3] = 1.5
    z[4, 12345] = 30.0
    u = torch.rand(5, generator=g, device="cuda")
    y, w = _labels(5, V, g)
    y[4], w[4] = 12345, 1.0
    for s in [dict(), dict(p=0.9), dict(k=300000, t=0.7), dict(k=700000, p=0.5), dict(m=0.2)]:
        _check_sample(cuda_lib, z, u, **s, what=str(s))
        _check_train(cuda_lib, z, y, w, **s, what=str(s))


def test_offsets_beyond_32_bits(cuda_lib):
    """More than 2^31 logits: the last rows give what they give alone."""
    T, V = 14500, 151936
    z = torch.empty(T, V, dtype=BF16, device="cuda")
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    z[-40:] *= 3.0
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.rand(T, generator=g, device="cuda")
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    s = (0.5, 30, 0.9, 0.0)
    tok, lp = cuda_lib.sample(z, u, *s)
    stats = cuda_lib.filtered_forward(z, y, *s)
    tok2, lp2 = cuda_lib.sample(z[-40:].clone(), u[-40:], *s)
    stats2 = cuda_lib.filtered_forward(z[-40:].clone(), y[-40:], *s)
    assert torch.equal(tok[-40:], tok2) and torch.equal(lp[-40:], lp2)
    for a, b in zip(stats, stats2):
        assert torch.equal(a[-40:], b)
    y[:] = tok
    lp, ent, rs, tau, idx = cuda_lib.filtered_forward(z, y, *s)
    grad = cuda_lib.filtered_backward(z, y, None, rs, tau, idx, s[0])
    part = cuda_lib.filtered_backward(z[-40:].clone(), y[-40:], None, rs[-40:], tau[-40:],
                                      idx[-40:], s[0])
    assert torch.equal(grad[-40:], part) and float(part.float().abs().max()) > 0


def test_two_streams_at_once(cuda_lib):
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    z, g = _rows(64, 50021, BF16, 51, peak=8.0)
    z[::4] = _rows(16, 50021, BF16, 52)[0]
    u = torch.rand(64, generator=g, device="cuda")
    args = (1.0, 0, 0.9, 0.0)
    want = cuda_lib.sample(z, u, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(cuda_lib.sample(z, u, *args))
    torch.cuda.synchronize()
    for tok, lp in got:
        assert torch.equal(tok, want[0]) and torch.equal(lp, want[1])


def test_draws_follow_the_distribution(cuda_lib):
    """Equidistant uniforms: token v is drawn round(p_v n) times, to within one
    at each end of its interval."""
    V, n = 50, 4096
    z = torch.randn(1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    for s in [(1.0, 0, 1.0, 0.0), (0.6, 10, 0.9, 0.0)]:
        tok, _ = cuda_lib.sample(z.repeat(n, 1), u, *s)
        kept, _, _, _, e = oflt.kept_set(z[0].double().cpu().numpy(), *s)
        p = np.where(kept, e, 0) / e[kept].sum()
        got = torch.bincount(tok, minlength=V).cpu().numpy()
        assert np.all(np.abs(got - p * n) <= 1.0 + 1e-6)


def test_gradient_against_differences(cuda_lib):
    """d logprob / d z by central differences of the oracle in float64, on a
    row whose cut lies far from a change of the kept set."""
    V = 40
    z = torch.randn(1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    z = z.double().float().requires_grad_()
    t, k = 0.7, 12
    zi = z.detach()[0].double().cpu().numpy()
    kept, _, _, _, _ = oflt.kept_set(zi, t, k)
    y = torch.tensor([int(np.flatnonzero(kept)[3])], device="cuda")
    lp, ent = cuda_lib.filtered_policy_stats(z, y, t, k)
    assert not ent.requires_grad
    lp.sum().backward()
    h = 1e-5
    for v in range(V):
        a, b = zi.copy(), zi.copy()
        a[v] += h
        b[v] -= h
        d = (oflt.forward(a, int(y), t, k)["logprob"] - oflt.forward(b, int(y), t, k)["logprob"]) / (2 * h)
        assert abs(z.grad[0, v].item() - d) <= 1e-6, v


def test_without_filters_equals_the_policy_statistics(cuda_lib):
    """Temperature 1 and no filter: the distribution of forward / backward."""
    z, g = _rows(33, 10007, BF16, 21)
    y, w = _labels(33, 10007, g)
    lp, ent, rs = cuda_lib.forward(z, y, IGN)
    lp2, ent2, rs2, tau, idx = cuda_lib.filtered_forward(z, y)
    assert torch.allclose(lp, lp2, rtol=0, atol=1e-5) and torch.allclose(ent, ent2, rtol=0, atol=1e-5)
    assert torch.allclose(rs, rs2, rtol=0, atol=1e-5)
    assert bool((tau == -math.inf).all()) and bool((idx == 10006).all())
    d1 = cuda_lib.backward(z, y, w, rs, IGN).float()
    d2 = cuda_lib.filtered_backward(z, y, w, rs2, tau, idx).float()
    assert torch.allclose(d1, d2, rtol=2.0**-7, atol=1e-9)


def test_other_stream_and_graph(cuda_lib):
    """On a side stream, and captured: replays read the buffers' new contents."""
    z, g = _rows(5, 40009, BF16, 30, peak=10.0)
    u = torch.rand(5, generator=g, device="cuda")
    y = torch.randint(0, 40009, (5,), generator=g, device="cuda")
    args = (0.8, 60, 0.95, 0.0)
    want = cuda_lib.sample(z, u, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cuda_lib.sample(z, u, *args)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    cuda_lib.filtered_forward(z, y, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, lp = cuda_lib.sample(z, u, *args)
        stats = cuda_lib.filtered_forward(z, y, *args)
        grad = cuda_lib.filtered_backward(z, y, None, *stats[2:], args[0])
    for _ in range(2):
        z.copy_(_rows(5, 40009, BF16, 31, peak=10.0)[0])
        u.copy_(torch.rand(5, generator=g, device="cuda"))
        graph.replay()
        tok2, lp2 = cuda_lib.sample(z, u, *args)
        stats2 = cuda_lib.filtered_forward(z, y, *args)
        grad2 = cuda_lib.filtered_backward(z, y, None, *stats2[2:], args[0])
        torch.cuda.synchronize()
        assert torch.equal(tok, tok2) and torch.equal(lp, lp2) and torch.equal(grad, grad2)
        for a, b in zip(stats, stats2):
            assert torch.equal(a, b)


def test_rollout_scoring_and_update_together(cuda_lib):
    """The operators as an RL step uses them: tokens drawn under temperature
    and top-p, scored under the same distribution, the surrogate's weights, the
    logits' gradient, and clipping by its norm."""
    z, g = _rows(24, 20000, BF16, 40, peak=10.0)
    s = (0.8, 0, 0.9, 0.0)
    tok, mu = cuda_lib.sample(z, torch.rand(24, generator=g, device="cuda"), *s)
    lp, ent, rs, tau, idx = cuda_lib.filtered_forward(z, tok, *s)
    # the policy that drew the tokens scores them the same
    assert torch.allclose(lp, mu, rtol=0, atol=2e-6)
    assert bool(torch.isfinite(lp).all())
    adv = torch.randn(24, generator=g, device="cuda")
    loss, w = cuda_lib.clipped_surrogate(lp, mu, adv, tok)
    grad = cuda_lib.filtered_backward(z, tok, w, rs, tau, idx, s[0])
    before = oflt.grad_norm([to_oracle(grad)])
    norm, (clipped,) = cuda_lib.clip_grad_norm([grad.clone()], 0.5 * before)
    assert abs(norm.item() - before) <= 2.0**-23 * before
    after = cuda_lib.grad_norm([clipped]).item()
    assert abs(after - 0.5 * before) <= 2.0**-8 * before


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("V", [1, 7, 15, 16, 17, 40, 2047, 2049, 4095, 4097, 12301])
def test_any_alignment(cuda_lib, dtype, out_dtype, V):
    """Rows at every offset from a 16-byte boundary, even and odd strides, inside
    memory full of NaN: the bits of an aligned copy's results, and nothing
    written beside the gradient."""
    T = 3
    g = torch.Generator(device="cuda").manual_seed(V)
    y = torch.randint(V, (T,), generator=g, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    w = torch.randn(T, generator=g, device="cuda")
    z0 = (3 * torch.randn(T, V, generator=g, device="cuda")).to(dtype)
    even = (V + 15) // 8 * 8
    base = torch.empty(T, even, device="cuda", dtype=dtype)[:, :V].copy_(z0)

    def results(z, out):
        got = []
        for s in ((1.0, 0, 1.0, 0.0), (0.7, 9, 0.9, 0.0)):
            got += cuda_lib.sample(z, u, *s)
            st = cuda_lib.filtered_forward(z, y, *s)
            grad = cuda_lib.filtered_backward(z, y, w, *st[2:], s[0], out=out)
            got += [*st, grad.clone()]
        return got

    want = results(base, torch.empty(T, even, device="cuda", dtype=out_dtype)[:, :V])
    for off in range(8):
        for pad, out_off, out_pad in ((0, 0, 0), (1, off, 1), (8, 8 - off, 3), (5, 1, 8)):
            mem = torch.full((off + T * (V + pad) + 16,), math.nan, device="cuda", dtype=dtype)
            z = mem.as_strided((T, V), (V + pad, 1), off).copy_(z0)
            store = torch.full((out_off + T * (V + out_pad) + 16,), 7.0, device="cuda", dtype=out_dtype)
            out = store.as_strided((T, V), (V + out_pad, 1), out_off)
            for i, (a, b) in enumerate(zip(results(z, out), want, strict=True)):
                assert torch.equal(a, b), (off, pad, out_off, out_pad, i)
            out.fill_(7.0)
            assert bool((store == 7.0).all()), (off, pad, out_off, out_pad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [128, 129, 256, 257, 511, 1024, 1025, 4000, 16384, 16385, 40000])
def test_candidate_counts(cuda_lib, dtype, V):
    """From a handful of candidates to more than a block lists, few and many
    finite logits: against the oracle, and with the bits of larger batches,
    which other numbers of threads finish."""
    z, g = _rows(5, V, dtype, V)
    z[1] = _rows(1, V, dtype, V + 1, mask=0.97)[0]
    z[2] = _rows(1, V, dtype, V + 2, std=0.2)[0]
    z[3] = _rows(1, V, dtype, V + 3, mask=0.6)[0]
    u = torch.rand(5, generator=g, device="cuda")
    u[4] = 0.0
    y = z.float().argmax(1)
    w = torch.ones(5, device="cuda")
    for s in (dict(k=129), dict(k=255, p=0.97), dict(k=300), dict(k=700, p=0.999), dict(k=1023),
              dict(k=1030, m=1e-4), dict(p=0.5), dict(p=0.9), dict(m=0.003), dict(p=0.999, m=0.001)):
        tok, lp = _check_sample(cuda_lib, z, u, what=(V, s), **s)
        stats = _check_train(cuda_lib, z, y, w, what=(V, s), **s)[:5]
        a = (1.0, s.get("k", 0), s.get("p", 1.0), s.get("m", 0.0))
        for n in (62, 124):  # 310 and 620 rows
            many = z.repeat(n, 1)
            tok2, lp2 = cuda_lib.sample(many, u.repeat(n), *a)
            assert torch.equal(tok2, tok.repeat(n)) and torch.equal(lp2, lp.repeat(n)), (V, s)
            for x, x2 in zip(stats, cuda_lib.filtered_forward(many, y.repeat(n), *a)):
                assert torch.equal(x2, x.repeat(n, *[1] * (x.dim() - 1))), (V, s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [0.3, 0.1, 0.03, 0.004])
def test_low_temperatures(cuda_lib, dtype, t):
    """top-k far below the maximum: tokens of weights from 2^-64 down to none are
    still counted, kept and, at u = 0, drawn."""
    for V in (2318, 20011, 60000):
        z, g = _rows(6, V, dtype, V, peak=12.0)
        z[3] = _rows(1, V, dtype, V + 1, peak=40.0)[0]
        u = torch.rand(6, generator=g, device="cuda")
        u[5] = 0.0
        w = torch.ones(6, device="cuda")
        y = z.float().topk(60, dim=1).indices[:, [0, 1, 7, 30, 49, 59]].diagonal().contiguous()
        for s in (dict(k=50), dict(k=200, p=0.95), dict(k=50, p=0.8, m=0.05), dict(k=200, m=1e-30),
                  dict(k=7, p=0.999999), dict(p=0.95), dict(m=1e-37)):
            _check_sample(cuda_lib, z, u, t=t, what=(V, s), **s)
            _check_train(cuda_lib, z, y, w, t=t, what=(V, s), **s)
