"""GPU tests of what holds on every path of the products in 8 bits (which one a call takes follows its sizes).

Values are whole numbers by powers of two, whose products and sums are exact in the instruction and in floats (below 2^24
steps), so results EQUAL the rounded reference's, formed in 64 bits on the GPU."""
import pytest
import torch

from tests.moe_testlib import say

pytestmark = pytest.mark.gpu
ops = pytest.importorskip("sparse_mixture_experts_level_amd.ops")
DEV = "cuda"


@pytest.mark.parametrize("hint,first", [(16, 2 ** 31 - 1 - 43), (128, 2 ** 31 - 1 - 300), (2 ** 31 - 1, 0)])
def test_rows_up_to_the_last_that_32_bits_count(hint, first):
    """Groups that end at row 2^31 - 1: of 43 and 300 rows announced as 16 and 128, whose last blocks of rows end within one
    block of 2^31, and one group of all rows, whose tiles are more than one launch takes."""
    R = 2 ** 31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    say(f"rows {first} to 2^31 - 1, announced as {hint}")
    x = torch.tensor([[1.0], [2.0], [-4.0], [0.5], [0.0]], device=DEV)
    codes, scale = ops.fp8_rows(5, 1)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    w8 = ops.fp8_weights(torch.tensor([[[3.0]], [[-2.0]]], device=DEV))
    off = torch.tensor([first, first + 20 if first else 0, R], dtype=torch.int32, device=DEV)
    index = torch.empty(R, dtype=torch.int32, device=DEV)
    y = torch.full((R, 1), 7.0, dtype=torch.bfloat16, device=DEV)
    step = 1 << 28
    for a in range(0, R, step):
        index[a:a + step] = torch.arange(a, min(a + step, R), device=DEV) % 5
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(2, R, hint, 1, 1))
    ops.moe_grouped_linear_fp8(2, R, hint, 1, 1, codes, scale, off, *w8, y, ws, row_index=index)
    torch.cuda.synchronize()
    del index
    for a in range(0, R, step):
        b = min(a + step, R)
        r = torch.arange(a, b, device=DEV)
        want = x[r % 5, 0] * torch.where(r < int(off[1]), 3.0, -2.0)
        want = torch.where(r < first, 7.0, want).bfloat16()
        assert torch.equal(y[a:b, 0], want), a
    del y, r, want
    torch.cuda.empty_cache()
