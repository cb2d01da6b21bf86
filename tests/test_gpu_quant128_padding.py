"""Codes past the end of a row or a group: zero, or NaN in a block that holds a NaN."""
import numpy as np
import pytest
import torch

import block128_reference as ref
from gpu_util import mxq
from test_gpu_quant128 import COLT, ROW, check, check_copy, spread, wide

pytestmark = pytest.mark.gpu


def nan_codes(codes):
    return (codes.cpu().numpy() & 0x7F) == 0x7F


@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_past_the_matrix(tile, dtype):
    x = spread((200, 300), 3, torch.bfloat16).to(dtype)
    x[190, 290] = float("nan")
    x[5, 299] = float("inf")
    got = mxq().quantize128(x, ROW | COLT, tile)
    check(got, x, tile, True)
    for codes, rows, (r, c) in ((got["q_row"], 200, (190, 290)), (got["q_colT"], 300, (290, 190))):
        nan = nan_codes(codes)
        K = codes.shape[1] - (84 if rows == 200 else 56)
        block = slice(r // tile * tile, min(r // tile * tile + tile, rows))
        assert nan[block, K:].all() and nan[block, K // 128 * 128:].all()  # the NaN's block, to its end
        rest = np.delete(codes.cpu().numpy(), np.r_[block], 0)[:, K:]
        assert not (rest & 0x7F).any()  # (zeros; an infinity's block too)


def test_past_a_group():
    sizes, C = [70, 200, 30], 140
    x = spread((sum(sizes), C), 4, torch.bfloat16)
    x[265, 7] = float("nan")  # in the second block of the second group
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    got = mxq().quantize128_grouped(x, ends)
    at = before = 0
    for n in sizes:
        codes = got["q_colT"][:, before:before + ref.up(n)]
        check_copy(codes, got["s_colT"][before // 128:(before + ref.up(n)) // 128], np.ascontiguousarray(wide(x[at:at + n]).T), 1, True)
        nan = nan_codes(codes)
        assert not np.delete(nan, 7, 0).any() and not nan[7, :128].any() and (n != 200 or nan[7, 128:].all())
        assert not (np.delete(codes.cpu().numpy(), 7, 0)[:, n:] & 0x7F).any()
        at, before = at + n, before + ref.up(n)
