"""The 8-bit head where the columns are an odd number of blocks of 128 and a CTA has
several tiles: the last block of a tile and the first of the next.  Against float64, with the
tolerance of test_gpu_fp8.py, and each row's bits against those of the whole batch."""
import pytest
import torch

from test_gpu_fp8 import BF16, F32, _check, _head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("K", [128, 384, 896])
@pytest.mark.parametrize("T", [1, 20, 64, 128])
def test_several_tiles(cuda_lib, T, K, out):
    q, s, W, Ws = _head(T, 40000, K, T + K)
    err = cuda_lib.new_error_flag("cuda:0")
    got = cuda_lib.fp8_logits(q, s, W, Ws, out, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    _check(got, q, s, W, Ws)
    for v in (0, 128 * 152, 39936):  # tiles of a CTA alone
        part = cuda_lib.fp8_logits(q, s, W[v:v + 128], Ws[v // 128:v // 128 + 1], out)
        assert torch.equal(part, got[:, v:v + 128])
