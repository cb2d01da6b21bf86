"""Arguments of the block-128 and Muon binding that it has to refuse before anything runs."""
import ctypes

import numpy as np
import pytest

from moe_grouped_gemm_mxq_amd import mxq
from test_block128_muon_refusals import (DEVICE, ENDS, HAS_GPU, ORTHOGONALIZE, SA, SB, SKB, SW, A, B, KB, W, call, dev,  # noqa: F401
                                         library, refused)  # (library: a fixture)


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


# (the first: 1.25 goes to -1.25, and what is above it grows with a slope of 24; the other with one of 1.4)
GROWING = [(-4.125, 11.375, -6.0), (1.0, -0.1201, 0.0768)]
STEADY = [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (1.0, 0.0, 0.0), (-1.0, 0.0, 0.0), (0.0, 0.0, 0.0)]


def orthogonalize_with(a, b, c):
    cfg = mxq.newton_schulz(coefficients=(a, b, c))
    return call("mxq_orthogonalize", ORTHOGONALIZE, dict(cfg=ctypes.byref(cfg)))


@pytest.mark.parametrize("coefficients", GROWING)
def test_coefficients_that_let_roundings_grow(coefficients):
    s = np.linspace(0, 1.25, 100001)
    a, b, c = coefficients
    assert np.abs(a * s + b * s ** 3 + c * s ** 5).max() <= 1.25 and abs(a + b * 1.255 ** 2 + c * 1.255 ** 4) > 1
    refused(orthogonalize_with(*coefficients), "grow")


@pytest.mark.parametrize("coefficients", STEADY)
def test_coefficients_that_do_not(coefficients):
    if HAS_GPU:
        pytest.skip("a GPU is present; this checks the no-device path")
    assert orthogonalize_with(*coefficients) == DEVICE


# 3 s - 1.5 s^3 reaches 1.63 at s = 0.82, whatever little is added
@pytest.mark.parametrize("coefficients", [(3.0, -1.5, 0.0), (3.0, -1.5, 1e-3), (3.0, -1.5, 1e-18), (3.0, -1.5, -1e-18), (-3.0, 1.5, 1e-18), (-3.0, 1.5, -1e-300),
                                          (3.0, -1e-18, -1.2), (3.0, 0.0, -1.2)])
def test_coefficients_that_pass_the_bound_within(coefficients):
    s = np.linspace(0, 1.25, 100001)
    a, b, c = coefficients
    assert np.abs(a * s + b * s ** 3 + c * s ** 5).max() > 1.25
    refused(orthogonalize_with(*coefficients), "coefficients")
