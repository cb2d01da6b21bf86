"""How far orthogonalised matrices are from 64 bits, by the figures that include/mxq.h states."""
import numpy as np
import pytest
import torch

import muon_reference as ref
from gpu_util import mxq
from test_gpu_muon import inputs, off, wide

pytestmark = pytest.mark.gpu


def matrices(kind, shape, seed):
    """noise, low_rank, decay, or noise with one row and one column `outliers_N` times as large."""
    if not kind.startswith("outliers"):
        return inputs(kind, shape, seed)
    x = inputs("noise", shape, seed)
    times = float(kind.split("_")[1])
    x[..., shape[-2] // 3, :] *= times
    x[..., :, shape[-1] // 2] *= times
    return x


def in_fp32(u, steps=5, coefficients=ref.COEFFICIENTS, eps=1e-7):
    """The same iteration in fp32 on the host, from a start that is rounded once."""
    a, b, c = (np.float32(v) for v in coefficients)
    x = (u / (np.sqrt((u * u).sum()) + eps)).astype(np.float32)
    if x.shape[0] > x.shape[1]:
        x = np.ascontiguousarray(x.T)
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return (x.T if u.shape[0] > u.shape[1] else x).astype(np.float64)


KINDS = ["noise", "low_rank", "decay", "outliers_100", "outliers_1000"]
SHAPES = [(5, 3), (8, 8), (16, 64), (64, 64), (64, 256), (300, 200), (3, 40, 100)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_fp32_results_are_as_near_as_fp32s(shape, kind):
    """Operands in 22 bits, where fp32 has 24: every rounding is at most four times that of the iteration in fp32, whose own
    distance is taken here; 2^-20 of it where that comes out small by chance (fp32's roundings, sixteen of them)."""
    for seed in range(3):
        x = matrices(kind, shape, seed)
        got = wide(mxq().orthogonalize(x, dtype=torch.float32)).reshape(-1, *shape[-2:])
        for a, u in zip(got, wide(x).reshape(-1, *shape[-2:])):
            want = ref.orthogonalize(u)
            e, single = off(a, want), off(in_fp32(u), want)
            print(shape, kind, seed, e, single, flush=True)
            assert e <= 4 * (single + 2.0 ** -20), (seed, e, single)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_bf16_results(shape, kind):
    """2^-9 for 64 rows and columns and more without outliers, 2^-6 otherwise; and the rounding to bf16."""
    stated = 2.0 ** -9 if min(shape[-2:]) >= 64 and not kind.startswith("outliers") else 2.0 ** -6
    for seed in range(3):
        x = matrices(kind, shape, seed)
        got = wide(mxq().orthogonalize(x)).reshape(-1, *shape[-2:])
        for a, u in zip(got, wide(x).reshape(-1, *shape[-2:])):
            e = off(a, ref.orthogonalize(u))
            print(shape, kind, seed, e, flush=True)
            assert e <= stated + 2.0 ** -8, (seed, e)


@pytest.mark.parametrize("steps,bf16,fp32", [(5, 2.0 ** -9, 2.0 ** -17), (8, 2.0 ** -8, 2.0 ** -17), (12, 2.0 ** -7, 2.0 ** -16), (32, 2.0 ** -5, 2.0 ** -13)])
def test_errors_grow_with_the_steps(steps, bf16, fp32):
    """The default coefficients do not converge: where the polynomial's slope is above 1, a step multiplies what is off."""
    x = inputs("noise", (128, 256), 7)
    want = ref.orthogonalize(wide(x), steps)
    for dtype, stated, rounding in ((torch.bfloat16, bf16, 2.0 ** -8), (torch.float32, fp32, 2.0 ** -24)):
        e = off(wide(mxq().orthogonalize(x, steps=steps, dtype=dtype)), want)
        print(steps, dtype, e, flush=True)
        assert e <= stated + rounding, (steps, dtype, e)
