"""The norm's bits depend on the list's values, types and sizes, not on where its
tensors lie: views that start at any element against copies of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", [[1], [7], [9], [8191], [8193, 5], [100003], [300001, 40000, 3],
                                   [5001] * 40, [16385] * 60], ids=lambda s: f"{len(s)}x{max(s)}")
def test_same_bits_at_any_offset(cuda_lib, dtype, sizes):
    gen = torch.Generator(device="cuda").manual_seed(len(sizes) + max(sizes))
    for scale in (1.0, 1e-12, 1e-30, 1e25, None):
        xs = []
        for n in sizes:
            x = torch.randn(n, generator=gen, device="cuda")
            if scale is None:  # of every size, and zeros
                x *= 10.0 ** torch.randint(-30, 15, (n,), generator=gen, device="cuda")
                x[::3] = 0.0
            xs.append((x if scale is None else x * scale).to(dtype))
        want = cuda_lib.grad_norm(xs)
        limit = want.item() * 0.5
        scaled = [torch.empty_like(x) for x in xs]
        cuda_lib.clip_grad_norm(xs, limit, out=scaled)
        for off in (1, 2, 3, 5, 7):
            views = []
            for i, x in enumerate(xs):
                o = (off + i) % 8
                store = torch.full((x.numel() + 16,), float("nan"), device="cuda", dtype=dtype)
                views.append(store[o:o + x.numel()].copy_(x))
            assert torch.equal(cuda_lib.grad_norm(views), want), (scale, off)
            norm, _ = cuda_lib.clip_grad_norm(views, limit)
            assert torch.equal(norm, want)
            assert all(torch.equal(a, b) for a, b in zip(views, scaled)), (scale, off)
