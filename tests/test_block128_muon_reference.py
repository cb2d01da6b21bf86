"""What pins the 64-bit references of the block-128 and Muon tests: torch's E4M3 type, exact fractions, singular values."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import block128_reference as ref
import muon_reference as muon


def test_values_of_the_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.TABLE, want, equal_nan=True)


def test_nearest_codes_are_torchs():
    steps = ref.TABLE[:127]
    middles = (steps[1:] + steps[:-1]) / 2  # ties, and their neighbours in fp32
    y = np.concatenate([steps, middles, np.nextafter(middles.astype(np.float32), np.float32(np.inf)).astype(np.float64),
                        np.nextafter(middles.astype(np.float32), np.float32(0)).astype(np.float64), np.random.default_rng(0).uniform(0, 448, 20000)])
    y = np.concatenate([y, -y]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_code(y.astype(np.float64)), want)


@pytest.mark.parametrize("shape", [(1, 1), (3, 130), (140, 129), (129, 300)])
@pytest.mark.parametrize("tile", [1, 128])
def test_quantiser_in_fractions(shape, tile):
    r = np.random.default_rng(sum(shape))
    x = torch.from_numpy(r.standard_normal(shape) * np.exp2(r.integers(-8, 9, (shape[0], 1)))).to(torch.bfloat16).double().numpy()
    x[0, 0] = 0.0
    codes, scales = ref.quantize(x, tile)
    R, C = shape
    assert codes.shape == (R, ref.up(C)) and scales.shape == (ref.up(C) // 128, -(-R // tile)) and not codes[:, C:].any()
    table = [Fraction(v) for v in ref.TABLE[:127]]
    for i in {0, R // 2, R - 1}:
        for b in range(ref.up(C) // 128):
            rows = slice(i // tile * tile, min(i // tile * tile + tile, R))
            amax = max([Fraction(abs(v)) for v in x[rows, b * 128:(b + 1) * 128].ravel()] + [Fraction(ref.FLOOR)])
            assert abs(Fraction(float(scales[b, i // tile])) - amax / 448) <= amax / 448 * Fraction(1, 2 ** 24)
            for k in range(b * 128, min(b * 128 + 128, C), 7):
                y = abs(Fraction(x[i, k])) * 448 / amax
                best = min(range(127), key=lambda c: (abs(table[c] - y), c & 1))
                assert codes[i, k] & 127 == best and bool(codes[i, k] >> 7) == bool(np.signbit(x[i, k]))


def test_a_groups_copy_is_its_transposes():
    r = np.random.default_rng(1)
    x, sizes = r.standard_normal((300, 40)), [0, 130, 1, 0, 169]
    codes, scales = ref.quantize_grouped(x, sizes)
    assert codes.shape == (40, sum(ref.up(m) for m in sizes)) and scales.shape == (codes.shape[1] // 128, 40)
    q, s = ref.quantize(np.ascontiguousarray(x[131:300].T))
    assert np.array_equal(codes[:, -256:], q) and np.array_equal(scales[-2:], s)
    assert np.abs(ref.values(codes, scales)[:, 256:257] - x[130:131].T).max() <= np.abs(x[130]).max() * 2.0 ** -4


def test_products_are_the_values():
    r = np.random.default_rng(2)
    A, sA = ref.quantize(r.standard_normal((5, 256)))
    B, sB = ref.quantize(r.standard_normal((140, 256)), 128)
    want, f32, bf16 = ref.product_and_bounds(A, sA, B, sB)
    a = torch.from_numpy(A).view(torch.float8_e4m3fn).double() * torch.from_numpy(sA).double().T.repeat_interleave(128, 1)
    b = torch.from_numpy(B).view(torch.float8_e4m3fn).double() * torch.from_numpy(sB).double().T.repeat_interleave(128, 0)[:140].repeat_interleave(128, 1)
    assert np.abs(want - (a @ b.T).numpy()).max() <= 1e-12 * np.abs(want).max()
    assert (f32 > 0).all() and (bf16 > f32).all()


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6)])
def test_iterations_act_on_singular_values(shape):
    x = np.random.default_rng(3).standard_normal(shape)
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    t = s / (np.linalg.norm(s) + 1e-7)
    for _ in range(5):
        t = 3.4445 * t - 4.7750 * t ** 3 + 2.0315 * t ** 5
    assert np.allclose(muon.orthogonalize(x), (u * t) @ vt, rtol=0, atol=1e-12)


@pytest.mark.parametrize("nesterov", [True, False])
def test_steps_are_the_lookahead_of_the_average(nesterov):
    """m' is an average with weight 1 - beta; nesterov's update is the average that would follow if g came again."""
    r = np.random.default_rng(4)
    p, g, m = (r.standard_normal((4, 6)) for _ in range(3))
    new, avg, o = muon.step(p, g, m, lr=0.1, momentum=0.8, nesterov=nesterov, weight_decay=0.5, scale=2.0, grad_scale=0.5)
    assert np.allclose(avg, m + 0.2 * (0.5 * g - m))
    u = avg + 0.2 * (0.5 * g - avg) if nesterov else avg
    assert np.allclose(o, muon.orthogonalize(u)) and np.allclose(new, 0.95 * p - 0.2 * o)
