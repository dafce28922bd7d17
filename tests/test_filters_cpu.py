"""Sampling, filtered statistics and gradient clipping without a GPU: the
oracle against brute force, and the argument checks of the C entry points and
of the Python layer (every call here fails validation; none launches)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import filters as oflt
from test_abi import _load


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("argument checks with made-up device pointers run only without a GPU")
    return _load()


# ---- the oracle ----------------------------------------------------------------

def _brute_kept(z, t, k, p, m):
    """The kept set by its definition, one token at a time."""
    V = len(z)
    order = sorted((v for v in range(V) if z[v] > -math.inf), key=lambda v: (-z[v], v))
    e = {v: math.exp((z[v] - z[order[0]]) / t) for v in order}
    if 0 < k < V:
        order = order[:k]
    if p < 1.0:
        total, run, out = math.fsum(e[v] for v in order), 0.0, []
        for v in order:
            out.append(v)
            run += e[v]
            if run >= p * total:
                break
        order = out
    return [v for v in order if e[v] >= m], e


@pytest.mark.parametrize("seed", range(20))
def test_oracle_against_brute_force(seed):
    rng = np.random.default_rng(seed)
    V = int(rng.integers(1, 60))
    z = rng.normal(size=V).round(1)
    z[rng.random(V) < 0.2] = -math.inf
    z[0] = 0.5
    t = float(np.float32(rng.choice([0.5, 1.0, 1.5])))
    k = int(rng.choice([0, 1, 5, 100]))
    p = float(np.float32(rng.choice([1.0, 0.31, 0.93])))
    m = float(np.float32(rng.choice([0.0, 0.13])))
    kept, tau, index, x, e = oflt.kept_set(z, t, k, p, m)
    want, eb = _brute_kept(z, t, k, p, m)
    assert sorted(np.flatnonzero(kept & np.isfinite(z))) == sorted(want)
    if math.isfinite(tau):
        assert index == want[-1] and tau == z[index]
        again = (z > tau) | ((z == tau) & (np.arange(V) <= index))
        assert np.array_equal(again, kept)
    S = math.fsum(eb[v] for v in want)
    u = float(np.float32(rng.random()))
    v, lp, near = oflt.sample(z, u, t, k, p, m)
    assert v in want and math.isclose(lp, math.log(eb[v] / S), rel_tol=1e-12, abs_tol=1e-14)
    below = math.fsum(eb[w] for w in want if w < v)
    assert below <= u * S + 1e-12 and u * S < below + eb[v] + 1e-12
    f = oflt.forward(z, want[0], t, k, p, m)
    assert math.isclose(f["logprob"], math.log(eb[want[0]] / S), rel_tol=1e-12, abs_tol=1e-14)
    H = -math.fsum(eb[w] / S * math.log(eb[w] / S) for w in want)
    assert math.isclose(f["entropy"], H, rel_tol=1e-10, abs_tol=1e-12)


def test_oracle_norm():
    assert oflt.grad_norm([np.float32([3.0]), np.float32([4.0])]) == 5.0
    assert oflt.grad_norm([np.zeros(0, np.float32)]) == 0.0
    assert math.isclose(oflt.grad_norm([np.full(4, 1e30, np.float32)]), 2e30, rel_tol=1e-6)


# ---- refusals of the C entry points ------------------------------------------------

P = ctypes.c_void_p


def _f(temperature=1.0, top_p=1.0, min_p=0.0, top_k=0, **rows):
    from vocab_wide_token_gb300 import pstat

    f = pstat.Filters(temperature, top_p, min_p, top_k, None, None, None, None)
    for name, v in rows.items():
        setattr(f, name, v)
    return f


def _sample(lib, logits=0x1000, dt=1, T=4, V=100, ld=100, u=0x2000, f=None, tok=0x3000, lp=0x4000,
            ws=0x5000, ws_bytes=1 << 40, filters=True):
    f = f or _f()
    return lib.pstat_sample(P(logits), dt, T, V, ld, P(u), ctypes.byref(f) if filters else None,
                            P(tok), P(lp), P(ws), ws_bytes, None, None)


def _forward(lib, logits=0x1000, dt=1, T=4, V=100, ld=100, y=0x2000, f=None, lp=0x3000,
             ent=0x3000, rs=0x3000, tau=0x3000, idx=0x3000, ws=0x5000, ws_bytes=1 << 40):
    f = f or _f()
    return lib.pstat_filtered_forward(P(logits), dt, T, V, ld, P(y), -100, ctypes.byref(f), P(lp),
                                      P(ent), P(rs), P(tau), P(idx), P(ws), ws_bytes, None, None)


@pytest.mark.parametrize("call", [_sample, _forward])
def test_filter_argument_checks(lib, call):
    assert call(lib, dt=3) == -4
    assert call(lib, T=-1) == -2 and call(lib, V=0) == -2 and call(lib, ld=99) == -2
    assert call(lib, V=(1 << 20) + 1, ld=1 << 21) == -2
    assert call(lib, T=(1 << 24) + 1) == -2
    assert call(lib, T=0, logits=0) == 0
    assert call(lib, logits=0) == -1
    assert call(lib, logits=0x1001) == -5 and call(lib, logits=0x1002, dt=0) == -5
    assert call(lib, lp=0) == -1 and call(lib, lp=0x3002) == -5
    for bad in (dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=2.0**21),
                dict(temperature=2.0**-21), dict(top_p=0.0), dict(top_p=1.5), dict(top_p=math.nan),
                dict(min_p=-0.1), dict(min_p=1.1), dict(min_p=math.nan)):
        assert call(lib, f=_f(**bad)) == -9, bad
    assert call(lib, ws=0) == -6 and call(lib, ws_bytes=64) == -6 and call(lib, ws=0x5008) == -5
    for rows in ("temperatures", "top_ks", "top_ps", "min_ps"):
        assert call(lib, f=_f(**{rows: 0x6002})) == -5, rows


def test_sample_argument_checks(lib):
    assert _sample(lib, filters=False) == -1
    assert _sample(lib, u=0) == -1 and _sample(lib, u=0x2002) == -5
    assert _sample(lib, tok=0) == -1 and _sample(lib, tok=0x3004) == -5


def test_filtered_forward_argument_checks(lib):
    for out in ("ent", "rs", "tau", "idx"):
        assert _forward(lib, **{out: 0}) == -1, out
    assert _forward(lib, y=0x2004) == -5 and _forward(lib, rs=0x3004) == -5
    assert _forward(lib, idx=0x3004) == -5
    assert _forward(lib, f=_f(temperature=0.0)) == -9  # no gradient at temperature 0


def test_filtered_backward_argument_checks(lib):
    def bwd(logits=0x1000, dt=1, T=4, V=100, ld=100, y=0x2000, w=0x2000, rs=0x3000, tau=0x3000,
            idx=0x3000, t=1.0, tt=0, out=0x4000, out_dt=1, ld_out=100):
        return lib.pstat_filtered_backward(P(logits), dt, T, V, ld, P(y), -100, P(w), P(rs),
                                           P(tau), P(idx), t, P(tt), P(out), out_dt, ld_out, None,
                                           None)
    assert bwd(dt=2) == -4 and bwd(dt=1, out_dt=0) == -4
    assert bwd(V=0) == -2 and bwd(ld=99) == -2 and bwd(ld_out=99) == -2 and bwd(T=-1) == -2
    assert bwd(T=0) == 0
    assert bwd(t=0.0) == -9 and bwd(t=math.nan) == -9
    for name in ("logits", "rs", "tau", "idx", "out"):
        assert bwd(**{name: 0}) == -1, name
    assert bwd(rs=0x3004) == -5 and bwd(tau=0x3002) == -5 and bwd(idx=0x3004) == -5
    assert bwd(y=0x2004) == -5 and bwd(w=0x2002) == -5 and bwd(tt=0x2002) == -5
    assert bwd(out=0x4001) == -5
    # the gradient may not go where the logits are (4 rows of 100 bf16 = 800 bytes)
    assert bwd(out=0x1000) == -9 and bwd(out=0x131E) == -9 and bwd(out=0x0CE2) == -9
    assert bwd(out=0x1320) in (-7, -8) and bwd(out=0x0CE0) in (-7, -8)


def test_filter_workspace_size(lib):
    n = ctypes.c_size_t(0)
    assert lib.pstat_filter_workspace_size(8, 1000, 1, ctypes.byref(n)) == 0
    assert lib.pstat_filter_workspace_size(8, 1000, 1, None) == -1
    assert lib.pstat_filter_workspace_size(8, 1000, 7, ctypes.byref(n)) == -4
    assert lib.pstat_filter_workspace_size(-1, 1000, 1, ctypes.byref(n)) == -2
    assert lib.pstat_filter_workspace_size(8, (1 << 20) + 1, 1, ctypes.byref(n)) == -2


def test_grad_argument_checks(lib):
    def words(*tensors):
        import array

        return array.array("q", [x for t in tensors for x in t])

    def norm(w, out=0x1000, ws=0x2000, ws_bytes=1 << 30):
        at = w.buffer_info()[0] if w is not None else None
        return lib.pstat_grad_norm(at, len(w) // 4 if w is not None else 1, P(out), P(ws), ws_bytes,
                                   None, None)

    def clip(w, limit=1.0):
        return lib.pstat_clip_grad_norm(w.buffer_info()[0], len(w) // 4, limit, P(0x1000),
                                        P(0x2000), 1 << 30, None, None)

    good = (0x1000, 0x1000, 10, 0)
    assert norm(None) == -1
    assert norm(words(good), out=0) == -1 and norm(words(good), ws=0) == -6
    assert norm(words(good), ws_bytes=8) == -6
    assert norm(words(good), ws=0x2004) == -5 and norm(words(good), out=0x1002) == -5
    assert norm(words((0, 0, 10, 0))) == -1
    assert norm(words(good, (0x1000, 0x1000, -1, 0))) == -2
    assert norm(words((0x1000, 0x1000, (1 << 40) + 1, 0))) == -2
    assert norm(words((0x1000, 0x1000, 10, 5))) == -4
    assert norm(words((0x1002, 0x1002, 10, 0))) == -5 and norm(words((0x1001, 0x1001, 10, 1))) == -5
    assert clip(words(good), -1.0) == -9 and clip(words(good), math.nan) == -9
    assert clip(words((0x1000, 0, 10, 0))) == -1 and clip(words((0x1000, 0x1002, 10, 0))) == -5
    # outputs that overlap: the same tensor twice, a view into another, an input
    # of another entry, a shifted copy of its own input
    assert clip(words(good, good)) == -9
    assert clip(words((0x1000, 0x1000, 10, 0), (0x1014, 0x1014, 10, 0))) == -9
    assert clip(words((0x1000, 0x2000, 10, 0), (0x3000, 0x1000, 10, 0))) == -9
    assert clip(words((0x1000, 0x1004, 10, 0))) == -9
    # these pass the checks and end at the missing device: inputs may overlap
    ok = clip(words((0x1000, 0x2000, 10, 0), (0x1000, 0x3000, 10, 0), (0x4000, 0x4000, 0, 0)))
    assert ok in (-7, -8)
    n = ctypes.c_size_t(0)
    assert lib.pstat_grad_workspace_size(None, 0, ctypes.byref(n)) == 0
    assert lib.pstat_grad_workspace_size(None, 0, None) == -1
    assert lib.pstat_grad_workspace_size(None, -1, ctypes.byref(n)) == -2


def test_binding_refusals(lib):
    """The Python layer refuses what it cannot describe to the library."""
    from vocab_wide_token_gb300 import pstat

    cpu, T = torch.device("cpu"), 6
    z = torch.zeros(T, 10)
    with pytest.raises(ValueError):
        pstat.sample(z, torch.zeros(T))  # not a CUDA tensor
    with pytest.raises(ValueError):
        pstat.grad_norm([torch.zeros(3)])
    with pytest.raises(ValueError):
        pstat.grad_norm([])
    for bad in (torch.ones(T, dtype=torch.float64), torch.ones(T + 1), torch.ones(T, 2)[:, 0]):
        with pytest.raises(ValueError):
            pstat._filters(bad, 0, 1.0, 0.0, T, cpu)
    with pytest.raises(ValueError):
        pstat._filters(1.0, torch.ones(T, dtype=torch.int64), 1.0, 0.0, T, cpu)
    f = pstat._filters(0.5, 7, 0.9, torch.zeros(T), T, cpu)._obj
    assert f.temperature == 0.5 and f.top_k == 7 and f.min_ps and not f.top_ps
    with pytest.raises(ValueError):
        pstat._filtered_outputs((torch.empty(T), torch.empty(T), torch.empty(T, 2), torch.empty(T),
                                 torch.empty(T)), T, cpu)
