"""Arguments of the block-128 and Muon binding that it has to refuse before anything runs."""
import pytest
import torch

from moe_grouped_gemm_mxq_amd import mxq
from test_block128_muon_refusals import ENDS, SA, SB, SKB, SW, A, B, KB, U8, W, dev, library  # noqa: F401  (library: a fixture)


def more(t):
    """The same under one more dim of three."""
    return dev(3, *t.shape)


@pytest.mark.parametrize("name,call", {
    "rows": lambda: mxq.gemm128(A, more(SA), B, SB),
    "tiles": lambda: mxq.gemm128(A, SA, B, more(SB)),
    "rows of experts' rows": lambda: mxq.grouped_gemm128(0, A, more(SA), W, SW, ENDS),
    "along tokens": lambda: mxq.mxq_grouped_gemm128(1, A, SA, KB, more(SKB), dev(2, 5, 300), ENDS),
}.items())
def test_scales_of_more_dims(name, call, library):  # noqa: F811
    with pytest.raises(ValueError, match="must be"):
        call()
    assert not library
