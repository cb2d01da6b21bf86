"""Newton-Schulz orthogonalisation and the Muon step against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import muon_reference as ref
from gpu_util import mxq

pytestmark = pytest.mark.gpu

# How far a result may be from the exact one, as a 2-norm relative to its own.  Every rounding of X to 22 bits, of an
# operand to fp16's 11 bits (a relative error of at most 2^-12 each, spread over independent elements) is multiplied by up
# to 3.4445 in each iteration left, but a relative error of X in directions that grow is a relative error of the result
# still.  Single products: six roundings an iteration of at most 2^-12 over five iterations, against factors of the last
# two (|b| s^2 and 2 c s^4 about 5) stay within 30 * 2^-12 / 2 = 3.7e-3; fp32 results with 2^-22 in the place of 2^-12 and
# fp32 sums over K: 30 * 2^-22 + (K / 16) 2^-23, times up to 3.4445^4 = 141 in directions that noise alone fills.
SINGLE = 4e-3
TRIPLE = 1e-4


def inputs(kind, shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    *lead, R, C = shape
    if kind == "noise":
        x = torch.randn(shape, generator=g)
    elif kind == "low_rank":
        k = max(1, min(R, C) // 16)
        x = torch.randn(*lead, R, k, generator=g) @ torch.randn(*lead, k, C, generator=g) + 0.01 * torch.randn(shape, generator=g)
    else:  # singular values falling as 1 / (i + 1)
        u, _, v = torch.linalg.svd(torch.randn(shape, generator=g), full_matrices=False)
        x = u @ (v / (torch.arange(min(R, C)) + 1.0)[:, None])
    return (x * 1e-3).to(dtype).cuda()


def wide(t):
    return t.detach().double().cpu().numpy()


def off(got, want):
    return np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)


def rounding(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


SHAPES = [(1, 1), (1, 64), (64, 1), (5, 3), (64, 64), (65, 130), (130, 65), (128, 256), (300, 200), (3, 100, 40), (2, 129, 257), (96, 700)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(shape, kind, dtype, out):
    x = inputs(kind, shape, len(shape), dtype)
    got = mxq().orthogonalize(x, dtype=out)
    assert got.shape == x.shape and got.dtype == out
    for a, b in zip(wide(got).reshape(-1, *shape[-2:]), wide(x).reshape(-1, *shape[-2:])):
        e = off(a, ref.orthogonalize(b))
        assert e <= (SINGLE if out == torch.bfloat16 else TRIPLE) + rounding(out), e


@pytest.mark.parametrize("steps,coefficients", [(1, ref.COEFFICIENTS), (2, ref.COEFFICIENTS), (8, ref.COEFFICIENTS), (9, (2.0, -1.5, 0.5)),
                                                (6, (1.5, -0.5, 0.0)), (3, (1.0, 0.0, 0.0))])
def test_other_iterations(steps, coefficients):
    x = inputs("decay", (70, 200), 5)
    want = ref.orthogonalize(wide(x), steps, coefficients)
    for out, tol in ((torch.bfloat16, SINGLE), (torch.float32, TRIPLE)):
        got = mxq().orthogonalize(x, steps=steps, coefficients=coefficients, dtype=out)
        assert off(wide(got), want) <= tol + rounding(out)


def test_extremes():
    m = mxq()
    for scale in (1e-30, 1e30):  # squares leave fp32's range
        x = inputs("noise", (40, 90), 1) * scale
        assert off(wide(m.orthogonalize(x, eps=0.0, dtype=torch.float32)), ref.orthogonalize(wide(x), eps=0.0)) <= TRIPLE
    x = inputs("noise", (3, 40, 90), 2)
    x[0] = 0
    x[2, 3, 5] = float("nan")
    y = m.orthogonalize(x)
    assert bool((y[0] == 0).all()) and bool(torch.isnan(y[2]).all())
    assert off(wide(y[1]), ref.orthogonalize(wide(x[1]))) <= SINGLE + 2.0 ** -8
    one = torch.zeros(200, 300, device="cuda")  # a single element: the largest that X has
    one[7, 9] = 3.0
    assert off(wide(m.orthogonalize(one, dtype=torch.float32)), ref.orthogonalize(wide(one))) <= TRIPLE
    assert m.orthogonalize(torch.zeros(0, 5, 6, device="cuda")).shape == (0, 5, 6)


def test_singular_values():
    x = inputs("noise", (128, 512), 3)
    s = np.linalg.svd(wide(mxq().orthogonalize(x)), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("param", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(96, 64), (40, 130), (3, 65, 70), (1, 7)])
def test_step(shape, nesterov, grad, param):
    m = mxq()
    p, g, mom = (0.02e3 * inputs("noise", shape, 1)).to(param), inputs("low_rank", shape, 2, grad), inputs("noise", shape, 3)
    copy = torch.zeros_like(p, dtype=torch.bfloat16) if param == torch.float32 else None
    h = dict(lr=2e-2, momentum=0.9, nesterov=nesterov, weight_decay=0.1, grad_scale=0.5)
    scale = m.muon_scale(shape)
    before = [wide(t).reshape(-1, *shape[-2:]) for t in (p, g, mom)]
    m.Muon([p], [g], [mom], copies=[copy]).step(**h)
    for i in range(before[0].shape[0]):
        want_p, want_m, o = ref.step(*(b[i] for b in before), scale=scale, **h)
        got_p, got_m = wide(p).reshape(-1, *shape[-2:])[i], wide(mom).reshape(-1, *shape[-2:])[i]
        # two products and a sum, each rounded; the terms may cancel
        size = 0.9 * np.abs(before[2][i]) + 0.1 * 0.5 * np.abs(before[1][i])
        assert np.all(np.abs(got_m - want_m) <= 4 * 2.0 ** -24 * size)
        tol = (SINGLE if param == torch.bfloat16 else TRIPLE) * h["lr"] * scale * np.linalg.norm(o)
        tol += (rounding(param) + 4 * 2.0 ** -24) * (np.linalg.norm(want_p) + h["lr"] * scale * np.linalg.norm(o))
        assert np.linalg.norm(got_p - want_p) <= tol
        if copy is not None:
            assert torch.equal(copy, p.to(torch.bfloat16))


def test_many_tensors_and_control():
    m = mxq()
    shapes = [(64, 32), (2, 40, 50), (130, 70)]
    make = lambda: ([20 * inputs("noise", s, 1) for s in shapes], [inputs("low_rank", s, 2) for s in shapes], [inputs("noise", s, 3) for s in shapes])  # noqa: E731
    a, b, c = make(), make(), make()
    m.Muon(*a).step(lr=0.01, grad_scale=0.25)
    m.Muon(*b).step(lr=99.0, grad_scale=99.0, control=m.adamw_control(0.01, 1, grad_scale=0.25))
    for x, y in zip(a[0] + a[2], b[0] + b[2]):
        assert torch.equal(x, y)
    opt, was = m.Muon(*c), [t.clone() for t in c[0] + c[2]]
    for lr, gs in ((float("nan"), 1.0), (0.01, float("inf"))):  # a step that is skipped changes nothing
        opt.step(lr=lr, grad_scale=gs)
        opt.step(control=m.adamw_control(lr, 1, grad_scale=gs))
    for x, y in zip(c[0] + c[2], was):
        assert torch.equal(x, y)
    m.Muon([], [], []).step()
