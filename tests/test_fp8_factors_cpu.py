"""The narrow 8-bit head's epilogue keeps a block's factors in one of two halves of shared
memory, written by a lane each and read by all.  Between a half's reads and its next write
lies the __syncwarp of the block between, so two blocks in a row, of one tile or
of two, may not have the same half.  Checked in the source: whether lanes run apart in
one build proves nothing."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "vocab_wide_token_gb300", "csrc", "fp8.cu")


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 7, 32])
def test_consecutive_blocks_have_different_halves(blocks):
    text = open(SOURCE).read()
    half, = re.findall(r"float\* fs = scales \+ \((\w+) & 1\) \* kCols;", text)
    body = text[text.index("float* fs = "):]
    assert body.count("fs[lane] = ", 0, body.index("tmem_load")) == 1
    assert body.index("fs[lane] = ") < body.index("__syncwarp();") < body.index("float4*>(fs")
    halves, it = [], 0
    for _ in range(5):  # a CTA's tiles
        for j in range(blocks):
            halves.append({"j": j, "it": it}[half] & 1)
            it += 1
    assert all(a != b for a, b in zip(halves, halves[1:]))
