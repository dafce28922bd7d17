"""The optimiser, the 8-bit head and the beam search without a GPU: the oracle against
direct statements of its parts, and the argument checks of the C entry points (every call
with made-up addresses fails validation, or at the missing device; none launches)."""
import ctypes
import itertools
import math
import struct

import numpy as np
import pytest
import torch

from oracle import adamw as oadam
from oracle import beams as obeams
from oracle import fp8 as ofp8
from test_abi import _load

P = ctypes.c_void_p
PASSED = (-7, -8)  # what a valid call comes to without a GPU


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("argument checks with made-up device pointers run only without a GPU")
    return _load()


# ---- the oracles ------------------------------------------------------------------

def test_oracle_e4m3_is_the_type():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ofp8.e4m3_values())
    x = np.concatenate([codes, (codes[1:] + codes[:-1]) / 2, -codes])
    want = torch.tensor(x).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ofp8.nearest(x), want)


def test_oracle_quantize():
    q, s = ofp8.quantize(np.array([[448.0] * 128 + [449.0] * 3 + [0.0]]), 1)
    assert s.tolist() == [[1.0, 2.0]] and q[0, 0] == 448 and q[0, 128] == 224
    q, s = ofp8.quantize(np.array([[0.0] * 130, [np.inf] + [1.0] * 129]), 1)
    assert s[0].tolist() == [1.0, 1.0] and math.isnan(s[1, 0]) and s[1, 1] == 2.0**-8
    assert not q[1, :128].any()


@pytest.mark.parametrize("seed", range(10))
def test_oracle_beams_against_all_continuations(seed):
    rng = np.random.default_rng(seed)
    B, beams, V, n = 2, int(rng.integers(1, 5)), int(rng.integers(1, 9)), int(rng.integers(1, 12))
    z = rng.normal(size=(B, beams, V)).round(1)
    z[rng.random(z.shape) < 0.3] = -np.inf
    scores = rng.normal(size=(B, beams))
    scores[0, 0] = -np.inf
    score, parent, token = obeams.select(z, scores, n)
    for b in range(B):
        every = []
        for k, v in itertools.product(range(beams), range(V)):
            row = z[b, k]
            if scores[b, k] > -np.inf and row[v] > -np.inf:
                every.append((scores[b, k] + row[v] - math.log(sum(math.exp(x) for x in row)), k, v))
        every.sort(key=lambda e: (-e[0], e[1:]))
        for i in range(n):
            if i >= len(every):
                assert (score[b, i], parent[b, i], token[b, i]) == (-np.inf, -1, -1)
            else:
                assert math.isclose(score[b, i], every[i][0], rel_tol=1e-12, abs_tol=1e-12)
                k, v = parent[b, i], token[b, i]
                assert math.isclose(next(e[0] for e in every if e[1:] == (k, v)), every[i][0],
                                    rel_tol=1e-12, abs_tol=1e-12)


@pytest.mark.parametrize("kind,step", [("m", 2.0**-3), ("v", 2.0**-3)])
def test_oracle_moments_by_block(kind, step):
    """Nearest codes are half a step off (2^-4 of the value), down to the block's depth."""
    rng = np.random.default_rng(3)
    x = np.float32(np.exp(rng.normal(size=300) * 2))
    if kind == "m":
        x *= np.where(rng.random(300) < 0.5, np.float32(-1), np.float32(1))
    state = oadam.encode(x, oadam.draws(None, 0, 300)[0], kind)
    got = oadam.decode(state, 300, kind)
    for b in range(3):
        at = slice(128 * b, min(300, 128 * b + 128))
        part = x[at].astype(np.float64)
        floor = 2.0 ** (np.floor(np.log2(np.abs(part).max())) - oadam.DEPTH[kind] + 1)
        deep = np.abs(part) >= floor
        assert deep.any() and (np.abs(got[at] - part)[deep] <= step / 2 * np.abs(part)[deep]).all()


def test_oracle_draws_are_even():
    """The draws of 4096 elements (32,768 for all eight steps): every bit of the 16 is set half the
    time, to 6 standard deviations of sqrt(n) / 2, alone, against its neighbours', and the
    parameter's against the moments'.  The two moments' draws, halves of one word, depend on
    one another: each is even, which is what keeps a moment's mean."""
    words = []
    for seed in range(8):
        m, v, p = oadam.draws(seed, seed // 2, 4096)
        words.append(np.stack([np.array(m) >> 4, np.array(v) >> 4, np.array(p)]))
    w = np.concatenate(words, axis=1)
    n = w.shape[1]
    for i in range(3):
        bits = w[i][:, None] >> np.arange(16) & 1
        assert (np.abs(bits.sum(0) - n / 2) <= 3 * math.sqrt(n)).all()
        same = (bits[1:] == bits[:-1]).sum(0)
        assert (np.abs(same - (n - 1) / 2) <= 3 * math.sqrt(n)).all()
    for i, j in ((0, 2), (1, 2)):
        same = ((w[i] ^ w[j])[:, None] >> np.arange(16) & 1).sum(0)
        assert (np.abs(same - n / 2) <= 3 * math.sqrt(n)).all()


# ---- refusals of the C entry points ---------------------------------------------------

def _tensors(rows):
    """pstat_adamw_tensor records as bytes: four addresses, n, two types, bits, padding."""
    return b"".join(struct.pack("<QQQQqiiii", *r) for r in rows)


def _step(lib, rows=None, n=None, options=True, **o):
    from vocab_wide_token_gb300 import pstat

    if rows is None:
        rows = [(0x10000, 0x20000, 0x30000, 0x40000, 100, 0, 0, 32, 0)]
    set_ = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, lr_at=None,
                step_at=None, seed_at=None, norm=None, seed=0, max_norm=0.0, random=0)
    set_.update(o)
    opt = pstat.AdamwOptions(**set_)
    return lib.pstat_adamw_step(_tensors(rows) if rows else None, len(rows) if n is None else n,
                                ctypes.byref(opt) if options else None, None, None)


def test_adamw_argument_checks(lib):
    good = [0x10000, 0x20000, 0x30000, 0x40000, 100, 0, 0, 32, 0]
    assert _step(lib) in PASSED
    assert _step(lib, options=False) == -1 and _step(lib, rows=[], n=1) == -1
    assert _step(lib, rows=[]) == 0
    assert _step(lib, n=-1) == -2 and _step(lib, n=(1 << 28) + 1) == -2

    def row(**at):
        r = list(good)
        for k, v in at.items():
            r[int(k[1:])] = v
        return _step(lib, rows=[r])
    for i in range(4):
        assert row(**{f"_{i}": 0}) == -1
        assert row(**{f"_{i}": good[i] + 2}) == -5
    assert row(_5=1, _0=0x10002) in PASSED and row(_6=1, _1=0x20002) in PASSED
    assert row(_7=8, _2=0x30001, _3=0x40001) in PASSED
    assert row(_5=2) == -4 and row(_6=3) == -4 and row(_7=16) == -4
    assert row(_4=-1) == -2 and row(_4=(1 << 40) + 1) == -2
    # overlaps: within a tensor, and of two tensors; shared gradients are none
    assert row(_0=0x20000) == -9 and row(_3=0x30000 + 396) == -9 and row(_3=0x30000 + 400) in PASSED
    assert row(_7=8, _3=0x30000 + 100) == -9 and row(_7=8, _3=0x30000 + 101) in PASSED
    assert _step(lib, rows=[good, good]) == -9
    assert _step(lib, rows=[good, [0x50000, 0x20000, 0x60000, 0x70000, 100, 0, 0, 32, 0]]) in PASSED
    assert _step(lib, rows=[good, [0, 0, 0, 0, 0, 0, 0, 32, 0]]) in PASSED


def test_adamw_option_argument_checks(lib):
    for bad in (dict(lr=-1.0), dict(lr=math.inf), dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf),
                dict(weight_decay=-1.0), dict(weight_decay=math.nan), dict(step=0), dict(step=-3),
                dict(norm=0x9000, max_norm=-1.0), dict(norm=0x9000, max_norm=math.nan)):
        assert _step(lib, **bad) == -9, bad
    for bad in (dict(lr_at=0x9002), dict(step_at=0x9004), dict(seed_at=0x9004), dict(norm=0x9002)):
        assert _step(lib, **bad) == -5, bad
    assert _step(lib, lr=math.nan, lr_at=0x9000, step=0, step_at=0x9000) in PASSED
    assert _step(lib, lr=0.0, eps=0.0, beta1=0.0, beta2=0.0) in PASSED


def test_adamw_moments_argument_checks(lib):
    def call(*rows, n=None):
        b = b"".join(struct.pack("<QQQQq", *r) for r in rows)
        return lib.pstat_adamw_moments(b or None, len(rows) if n is None else n, None)
    good = (0x10001, 0x20001, 0x30000, 0x40000, 129)
    assert call(good) in PASSED and call() == 0
    assert call(n=1) == -1 and call(good, n=-1) == -2
    for i in range(4):
        assert call(good[:i] + (0,) + good[i + 1:]) == -1
    assert call(good[:2] + (0x30002,) + good[3:]) == -5
    assert call(good[:4] + (-1,)) == -2
    assert call(good, good) == -9 and call(good, (0x10001, 0x20001, 0x50000, 0x60000, 129)) in PASSED
    assert call((0x10001, 0x20001, 0x10000, 0x40000, 129)) == -9
    assert call((0, 0, 0, 0, 0)) in PASSED + (0,)


def _quantize(lib, x=0x1000000, dt=1, T=4, K=256, ld=256, rows=1, q=0x2000000, s=0x3000000, sr=1, sc=4):
    return lib.pstat_fp8_quantize(P(x), dt, T, K, ld, rows, P(q), P(s), sr, sc, None, None)


def test_quantize_argument_checks(lib):
    assert _quantize(lib) in PASSED
    assert _quantize(lib, T=0, x=0) == 0
    assert _quantize(lib, dt=2) == -4
    for bad in (dict(T=-1), dict(K=0), dict(ld=255), dict(rows=2), dict(rows=0), dict(K=1 << 31, ld=1 << 31),
                dict(T=1 << 31), dict(sr=0), dict(sc=0), dict(sr=-1), dict(sc=(1 << 31) + 1),
                dict(sr=1, sc=1), dict(sr=1, sc=3), dict(T=1 << 30, K=1 << 30, ld=1 << 30, sc=1 << 30)):
        assert _quantize(lib, **bad) == -2, bad
    assert _quantize(lib, sr=2, sc=1) in PASSED and _quantize(lib, T=1, sr=1, sc=1) in PASSED
    assert _quantize(lib, rows=128, sr=1, sc=1) in PASSED and _quantize(lib, T=129, rows=128, sr=1, sc=1) == -2
    for name in ("x", "q", "s"):
        assert _quantize(lib, **{name: 0}) == -1
    assert _quantize(lib, x=0x1000001) == -5 and _quantize(lib, dt=0, x=0x1000002) == -5
    assert _quantize(lib, s=0x3000002) == -5 and _quantize(lib, q=0x2000003) in PASSED
    size = 4 * 256 * 2  # of x in bytes
    assert _quantize(lib, q=0x1000000 + size - 1) == -9 and _quantize(lib, q=0x1000000 + size) in PASSED
    assert _quantize(lib, s=0x1000000 + size - 4) == -9 and _quantize(lib, s=0x2000000) == -9
    assert _quantize(lib, ld=1 << 61, q=0x2000000) == -9  # saturates: reaches over everything


def _logits(lib, q=0x1000000, qs=0x2000000, sr=1, sc=4, W=0x3000000, ws=0x4000000, T=4, V=100, K=256,
            out=0x5000000, dt=1, ld=100):
    return lib.pstat_fp8_logits(P(q), P(qs), sr, sc, P(W), P(ws), T, V, K, P(out), dt, ld, None, None)


def test_logits_argument_checks(lib):
    assert _logits(lib) in PASSED and _logits(lib, T=0, q=0) == 0
    assert _logits(lib, dt=2) == -4
    for bad in (dict(T=-1), dict(V=0), dict(ld=99), dict(K=0), dict(K=250), dict(K=8), dict(K=(1 << 24) + 16),
                dict(T=1 << 30), dict(V=1 << 30, ld=1 << 30), dict(sr=-1), dict(sc=-1),
                dict(sr=(1 << 31) + 1)):
        assert _logits(lib, **bad) == -2, bad
    for name in ("q", "qs", "W", "ws", "out"):
        assert _logits(lib, **{name: 0}) == -1
    assert _logits(lib, q=0x1000008) == -5 and _logits(lib, W=0x3000008) == -5
    assert _logits(lib, qs=0x2000002) == -5 and _logits(lib, ws=0x4000002) == -5
    assert _logits(lib, out=0x5000001) == -5 and _logits(lib, dt=0, out=0x5000002) == -5
    assert _logits(lib, sr=0, sc=0) in PASSED  # one scale for all
    for at in (0x1000000, 0x1000000 + 1022, 0x2000000 + 28, 0x3000000 + 100 * 256 - 2, 0x4000000 + 4):
        assert _logits(lib, out=at) == -9, hex(at)
    assert _logits(lib, out=0x1000000 + 1024) in PASSED


def _beams(lib, z=0x1000000, dt=1, B=2, beams=3, V=100, ld=100, s=0x2000000, n=6, score=0x3000000,
           parent=0x4000000, token=0x5000000, ws=0x6000000, ws_bytes=1 << 30):
    return lib.pstat_beam_select(P(z), dt, B, beams, V, ld, P(s), n, P(score), P(parent), P(token), P(ws),
                                 ws_bytes, None, None)


def test_beam_argument_checks(lib):
    need = ctypes.c_size_t(0)
    assert lib.pstat_beam_workspace_size(2, 3, 100, 1, None) == -1
    assert lib.pstat_beam_workspace_size(2, 3, 100, 1, ctypes.byref(need)) == 0 and need.value > 0
    assert lib.pstat_beam_workspace_size(2, 65, 100, 1, ctypes.byref(need)) == -2
    assert _beams(lib) in PASSED and _beams(lib, ld=0) in PASSED and _beams(lib, B=0, z=0) == 0
    assert _beams(lib, dt=2) == -4
    for bad in (dict(B=-1), dict(beams=0), dict(beams=65), dict(V=0), dict(V=(1 << 20) + 1, ld=1 << 21),
                dict(ld=99), dict(ld=-1), dict(n=0), dict(n=129), dict(B=(1 << 24) // 3 + 1)):
        assert _beams(lib, **bad) == -2, bad
    for name in ("z", "s", "score", "parent", "token"):
        assert _beams(lib, **{name: 0}) == -1
    assert _beams(lib, ws=0) == -6 and _beams(lib, ws_bytes=need.value - 1) == -6
    assert _beams(lib, ws_bytes=need.value) in PASSED
    for bad in (dict(z=0x1000001), dict(z=0x1000002, dt=0), dict(s=0x2000002), dict(score=0x3000002),
                dict(parent=0x4000004), dict(token=0x5000004), dict(ws=0x6000008)):
        assert _beams(lib, **bad) == -5, bad
    assert _beams(lib, score=0x2000000) == -9 and _beams(lib, score=0x2000000, n=3) in PASSED
    for bad in (dict(score=0x4000000), dict(parent=0x5000000), dict(token=0x6000000), dict(score=0x1000000),
                dict(ws=0x1000000), dict(s=0x6000000), dict(score=0x2000004, n=3)):
        assert _beams(lib, **bad) == -9, bad


def _reorder(lib, *states, parents=0x9000000, B=2, beams=3, out_beams=3, n=None):
    b = b"".join(struct.pack("<QQqqqqqq", *s) for s in states)
    return lib.pstat_beam_reorder(b or None, len(states) if n is None else n, P(parents), B, beams, out_beams,
                                  None, None)


def test_reorder_argument_checks(lib):
    #        data       out        rows      segments, strides, bytes
    plain = (0x1000000, 0x2000000, 64, 64, 1, 64, 64, 64)
    here = (0x1000000, 0x1000000, 64, 64, 1, 64, 64, 64)
    assert _reorder(lib, plain) in PASSED and _reorder(lib, here) in PASSED
    assert _reorder(lib) == 0 and _reorder(lib, plain, B=0) == 0
    for bad in (dict(B=-1), dict(beams=0), dict(beams=65), dict(out_beams=0), dict(out_beams=129), dict(n=-1)):
        assert _reorder(lib, plain, **bad) == -2, bad
    assert _reorder(lib, n=1) == -1
    assert _reorder(lib, plain, parents=0) == -1 and _reorder(lib, plain, parents=0x9000004) == -5
    assert _reorder(lib, (0,) + plain[1:]) == -1 and _reorder(lib, plain[:1] + (0,) + plain[2:]) == -1

    def change(base, **at):
        s = list(base)
        for k, v in at.items():
            s[int(k[1:])] = v
        return _reorder(lib, tuple(s))
    big = 1 << 46
    for bad in (dict(_4=-1), dict(_7=-1), dict(_2=-1), dict(_3=big + 1), dict(_4=big, _7=big), dict(_3=63),
                dict(_4=2, _6=63, _3=256), dict(_3=big), dict(_2=big), dict(_4=1 << 30, _6=1 << 30, _7=1)):
        assert change(plain, **bad) == -2, bad
    assert change(plain, _4=0) in PASSED + (0,) and change(plain, _7=0) in PASSED + (0,)
    # in place: for all states or none, equal strides, as many beams
    assert _reorder(lib, here, (0x3000000, 0x4000000) + plain[2:]) == -9
    assert _reorder(lib, here, out_beams=2) == -9 and change(here, _3=128) == -9
    assert change(here, _4=2, _5=32, _6=16, _7=16) == -9
    # overlaps
    assert change(plain, _1=0x1000000 + 6 * 64 - 1) == -9 and change(plain, _1=0x1000000 + 6 * 64) in PASSED
    assert _reorder(lib, plain, (0x3000000, 0x2000000) + plain[2:]) == -9
    assert _reorder(lib, plain, (0x1000000, 0x3000000) + plain[2:]) in PASSED  # one input twice
    assert _reorder(lib, here, here) == -9
    for at in (0x2000000, 0x2000000 + 376):  # the parents in an output
        assert _reorder(lib, plain, parents=at) == -9
    assert _reorder(lib, plain, parents=0x2000000 + 384) in PASSED
    assert _reorder(lib, plain, parents=0x1000000) in PASSED  # in an input
    # two halves of the rows of one buffer
    left, right = (0x1000000, 0x2000000, 128, 128, 1, 64, 64, 64), (0x1000040, 0x2000040, 128, 128, 1, 64, 64, 64)
    assert _reorder(lib, left, right) in PASSED
    assert _reorder(lib, left, right[:1] + (0x2000020,) + right[2:]) == -9
