"""Both marshalling paths of a call, the native module's and the one in Python
(taken here by switching the module off), give the same bits, and refuse the same."""
import pytest
import torch

from vocab_wide_token_gb300 import pstat

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture
def both(cuda_lib, monkeypatch):
    if pstat._native is None:
        pytest.fail("the native module is not built")

    def run(call):
        a = call()
        with monkeypatch.context() as m:
            m.setattr(pstat, "_native", None)
            b = call()
        return a, b

    return run


def same(a, b):
    for x, y in zip(a, b, strict=True):
        assert x.dtype == y.dtype and x.shape == y.shape and x.device == y.device
        assert torch.equal(x.contiguous().view(torch.uint8) if x.dim() else x.view(1).view(torch.uint8),
                           y.contiguous().view(torch.uint8) if y.dim() else y.view(1).view(torch.uint8))


def settings(T, per_row):
    if not per_row:
        return 0.8, 20, 0.9, 0.01
    i = torch.arange(T, device=DEV, dtype=torch.float32)
    return (0.5 + 0.1 * (i % 4), (3 + i % 5).to(torch.int32), 1 - 0.05 * (i % 3), 0.01 * (i % 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pad", [(1, 1, 0), (1, 1000, 0), (5, 333, 3), (9, 4096, 0), (0, 16, 0)])
@pytest.mark.parametrize("per_row", [False, True])
def test_filtered_calls(both, dtype, T, V, pad, per_row):
    gen = torch.Generator(DEV).manual_seed(5)
    z = torch.randn(T, V + pad, device=DEV, generator=gen).mul_(3).to(dtype)[:, :V]
    u = torch.rand(T, device=DEV, generator=gen)
    y = torch.randint(V, (T,), device=DEV, generator=gen)
    w = torch.randn(T, device=DEV, generator=gen)
    s = settings(T, per_row)
    same(*both(lambda: pstat.sample(z, u, *s)))
    for labels in (y, None):
        a, b = both(lambda: pstat.filtered_forward(z, labels, *s))
        same(a, b)
        for weights in (w, None):
            same(*both(lambda: (pstat.filtered_backward(z, labels, weights, *a[2:], s[0]),)))


@pytest.mark.parametrize("sizes", [[1], [0, 3], [5, 7, 100_000, 1]])
def test_gradient_calls(both, sizes):
    g = [torch.randn(n, device=DEV).to(torch.bfloat16 if i % 2 else torch.float32)
         for i, n in enumerate(sizes)]
    same(*both(lambda: (pstat.grad_norm(g),)))
    same(*both(lambda: (pstat.grad_norm(tuple(g)),)))

    def clip():
        out = [torch.empty_like(x) for x in g]
        norm, got = pstat.clip_grad_norm(g, 0.5, out=out)
        assert all(a is b for a, b in zip(got, out, strict=True))
        return (norm, *got)

    def clip_in_place():
        own = [x.clone() for x in g]
        norm, got = pstat.clip_grad_norm(own, 1)
        assert all(a is b for a, b in zip(got, own, strict=True))
        return (norm, *got)

    same(*both(clip))
    same(*both(clip_in_place))


def test_refusals(both):
    z = torch.randn(3, 64, device=DEV)
    u = torch.rand(3, device=DEV)
    y = torch.zeros(3, dtype=torch.int64, device=DEV)
    g = torch.randn(8, device=DEV)

    def refused(call):
        try:
            call()
        except (ValueError, TypeError, pstat.PstatError) as e:
            return type(e), str(e)
        pytest.fail("not refused")

    for call in (lambda: pstat.sample(z[:, ::2], u), lambda: pstat.sample(z.half(), u),
                 lambda: pstat.sample(z, u[:2]), lambda: pstat.sample(z, u.double()),
                 lambda: pstat.sample(z, u, -1.0), lambda: pstat.sample(z, u, 1.0, 0, 2.0),
                 lambda: pstat.sample(z, u, u[:2]), lambda: pstat.sample(z, u, "a"),
                 lambda: pstat.sample(z[:1].expand(3, 64), u),
                 lambda: pstat.sample(z, u, dev_error=u),
                 lambda: pstat.filtered_forward(z, y.int()),
                 lambda: pstat.filtered_forward(z, y, 0.0),
                 lambda: pstat.filtered_backward(z, y, None, z[:, :2], u, y),
                 lambda: pstat.filtered_backward(z, y, None, None, u, y),
                 lambda: pstat.grad_norm([g, g.half()]), lambda: pstat.grad_norm([g, g.cpu()]),
                 lambda: pstat.clip_grad_norm([g, g], 1.0),
                 lambda: pstat.clip_grad_norm([g], -1.0),
                 lambda: pstat.clip_grad_norm([g], 1.0, out=[g[:4]]),
                 lambda: pstat.clip_grad_norm([g], 1.0, out=[])):
        a, b = both(lambda: refused(call))
        assert a == b


def test_error_flags_and_large_top_k(both):
    z = torch.randn(2, 64, device=DEV)
    u = torch.tensor([0.5, 1.5], device=DEV)  # no uniform: flagged
    flags = [pstat.new_error_flag(z.device) for _ in range(2)]
    it = iter(flags)
    same(*both(lambda: pstat.sample(z, u, dev_error=next(it))))
    assert flags[0].item() == flags[1].item() != 0
    same(*both(lambda: pstat.sample(z, u[:1].expand(2).contiguous(), 1.0, 1 << 70)))


def test_another_stream_and_a_graph(both):
    z = torch.randn(4, 5000, device=DEV)
    u = torch.rand(4, device=DEV)
    want = pstat.sample(z, u, 1.0, 50, 0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pstat.sample(z, u, 1.0, 50, 0.9)
    torch.cuda.synchronize()
    same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pstat.sample(z, u, 1.0, 50, 0.9)
    graph.replay()
    torch.cuda.synchronize()
    same(got, want)


@pytest.mark.parametrize("before", ["nothing", "kernel", "copy", "memset", "join", "join of copies"])
def test_captured_behind(cuda_lib, before):
    """Captured calls behind whatever comes before them: what is written there is
    what they read, replay after replay."""
    T, V = 6, 5000
    src = [torch.randn(T, V, device=DEV), torch.rand(T, device=DEV)]
    z, u = torch.empty(T, V, device=DEV), torch.empty(T, device=DEV)
    y = torch.arange(T, device=DEV)
    w = torch.empty(T, device=DEV)
    side = torch.cuda.Stream()

    def feed():
        main = torch.cuda.current_stream()
        if before == "kernel":
            torch.mul(src[1], 1.0, out=u)
            w.fill_(1.0)
            torch.mul(src[0], 2.0, out=z)
        elif before == "copy":
            u.copy_(src[1])
            w.fill_(1.0)
            z.copy_(src[0])
        elif before == "memset":
            u.copy_(src[1])
            z.copy_(src[0])
            w.zero_()
        else:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                z.copy_(src[0]) if before.endswith("copies") else torch.mul(src[0], 2.0, out=z)
            w.fill_(1.0)
            u.copy_(src[1]) if before.endswith("copies") else torch.mul(src[1], 1.0, out=u)
            main.wait_stream(side)

    def calls():
        if before != "nothing":
            feed()
        got = list(pstat.sample(z, u, 0.9, 40, 0.9))
        if before != "nothing":
            feed()
        st = pstat.filtered_forward(z, y, 0.9, 40, 0.9)
        if before != "nothing":
            feed()
        got += [*st, pstat.filtered_backward(z, y, w, *st[2:], 0.9)]
        if before != "nothing":
            feed()
        big = [z, z[:1].reshape(-1), z.reshape(-1)[:7]] * 8
        return got + [pstat.grad_norm(big), pstat.grad_norm([z])]

    if before == "nothing":
        z.copy_(src[0]), u.copy_(src[1]), w.fill_(1.0)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        for x in src:
            x.copy_(torch.rand_like(x) if x.dim() == 1 else torch.randn_like(x))
        if before == "nothing":
            z.copy_(src[0]), u.copy_(src[1])
        graph.replay()
        torch.cuda.synchronize()
        same(got, calls())
