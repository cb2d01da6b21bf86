"""Matrices of zeros (experts without tokens) where eps does not keep the norm from zero."""
import pytest
import torch

import muon_reference as ref
from gpu_util import mxq
from test_gpu_muon import inputs, off, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-310, 1e-7])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(40, 70), (70, 40)])
def test_orthogonalize(shape, out, eps):
    x = inputs("noise", (3, *shape), 1)
    x[1] = 0
    y = mxq().orthogonalize(x, eps=eps, dtype=out)
    assert bool((y[1] == 0).all())
    for i in (0, 2):  # 2^-14 and 2^-6: see the header; and a rounding
        assert off(wide(y[i]), ref.orthogonalize(wide(x[i]), eps=eps)) <= (2.0 ** -6 + 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -14)


@pytest.mark.parametrize("eps", [0.0, 1e-310])
def test_step(eps):
    p, g, m = inputs("noise", (2, 40, 70), 1), inputs("noise", (2, 40, 70), 2), torch.zeros(2, 40, 70, device="cuda")
    g[1] = 0
    was = p.clone()
    mxq().Muon([p], [g], [m]).step(lr=0.1, weight_decay=0.5, eps=eps)
    assert off(wide(p[1]), 0.95 * wide(was[1])) <= 2.0 ** -23  # (1 - lr wd and the product rounded)
    assert bool(p.isfinite().all()) and not torch.equal(p[0], 0.95 * was[0])
