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


@pytest.mark.parametrize("shape", [(0, 40), (40, 0), (3, 0, 40), (0, 0, 4), (2 ** 20 + 1, 1), (65536, 1, 1)])
def test_weights_that_a_step_would_refuse(shape):
    """Named when the Muon is made: a step that came upon them would have updated the weights before."""
    mxq.mxq_orthogonalize_workspace.cache_clear()
    first = [dev(4, 4), dev(2, 4, 5)]
    with pytest.raises(ValueError, match=r"tensor 2: .*1 to 2\^20 .*65535"):
        mxq.Muon(*([*first, dev(*shape)] for _ in range(3)))
    assert len(mxq.Muon(first, first, first).tensors) == 2
    assert len(mxq.Muon([dev(0, 4, 4)], [dev(0, 4, 4)], [dev(0, 4, 4)]).tensors) == 1  # (no experts here)
