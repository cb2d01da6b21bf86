"""FP8 quantisers with a scale for each block of 128 against the 64-bit reference."""
import numpy as np
import pytest
import torch

import block128_reference as ref
from gpu_util import mxq

pytestmark = pytest.mark.gpu
ROW, COLT = 1, 2
GUARD = 0xA5


def wide(t):
    return t.detach().double().cpu().numpy()


def check_copy(codes, scales, x, tile, exact):
    """One copy against the row copy of x (64-bit host matrix)."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    want, want_s = ref.quantize(x, tile)
    assert np.array_equal(scales.view(np.uint32)[~np.isnan(want_s)], want_s.view(np.uint32)[~np.isnan(want_s)])
    assert np.array_equal(np.isnan(scales), np.isnan(want_s))
    if exact:
        assert np.array_equal(codes & 0x7F, want & 0x7F)
        finite = (want & 0x7F) != 0x7F
        assert np.array_equal(codes[finite], want[finite])
        return
    # fp32: the quotient is off by at most 2^-23 of itself before it is rounded
    y, v = ref.quotients(x, tile), ref.TABLE[codes]
    assert np.all(np.abs(v - y) <= ref.step_of(np.abs(y) * (1 + 2.0 ** -22)) / 2 + 2.0 ** -23 * np.abs(y))
    assert np.array_equal(codes >> 7, np.signbit(y).astype(np.uint8))


def check(got, x, tile, exact):
    """All copies in `got` of x [R][C] or [batch][R][C]."""
    mats = x if x.dim() == 3 else x[None]
    for name, turn in (("row", False), ("colT", True)):
        if "q_" + name not in got:
            continue
        q, s = got["q_" + name], got["s_" + name]
        for i, m in enumerate(mats):
            h = wide(m)
            check_copy(q[i] if x.dim() == 3 else q, s[i] if x.dim() == 3 else s, np.ascontiguousarray(h.T) if turn else h, tile, exact)


def spread(shape, seed, dtype):
    """Values over many binades, with zeros of both signs and a column and a row of zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-30, 30, (shape[0], 1), generator=g).float())
    x[torch.rand(shape, generator=g) < 0.05] = 0.0
    x[torch.rand(shape, generator=g) < 0.05] = -0.0
    if shape[0] > 2:
        x[shape[0] // 2] = 0.0
    if shape[1] > 2:
        x[:, shape[1] // 2] = -0.0
    return x.to(dtype).cuda()


SHAPES = [(1, 1), (1, 128), (7, 300), (16, 129), (128, 128), (129, 257), (300, 1000), (2, 7168), (1000, 3), (257, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("axes", [ROW, COLT, ROW | COLT])
@pytest.mark.parametrize("shape", SHAPES)
def test_copies(shape, axes, tile, dtype):
    x = spread(shape, sum(shape) + axes, dtype)
    got = mxq().quantize128(x, axes, tile)
    assert set(got) == {n for n, bit in (("q_row", ROW), ("s_row", ROW), ("q_colT", COLT), ("s_colT", COLT)) if axes & bit}
    check(got, x, tile, dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_bf16_ratio_rounds_as_the_exact_quotient(dtype):
    """Blocks whose largest values run over a binade's mantissas, against all mantissas: ties and their neighbours."""
    amax = torch.arange(128, 256).float()
    other = torch.cat([torch.arange(128, 256).float() * 2.0 ** -k for k in range(1, 13)]) * 0.5
    x = torch.zeros(128, 13 * 128)
    x[:, : other.numel()] = other
    x[:, 12 * 128:] = 0
    x = torch.cat([torch.minimum(x[:, b * 128:(b + 1) * 128], amax[:, None]) for b in range(12)], 1)
    x[:, ::128] = amax[:, None]
    x = x.to(dtype).cuda()
    got = mxq().quantize128(x)
    check(got, x, 1, True)  # (these fp32 values are bf16 values too)


@pytest.mark.parametrize("tile", [1, 128])
def test_batches_and_strides(tile):
    m = mxq()
    big = spread((5 * 140, 400), 3, torch.bfloat16).view(5, 140, 400)
    for x in (big, big[:, :131], big[1:4, 3:, :257], big[:, :, 1:300], big[::2, ::2, 8:], big[:0]):
        got = m.quantize128(x, ROW | COLT, tile)
        check(got, x, tile, True)
    flat = big[0]
    for x in (flat[:, 3:200], flat[::3], flat[1:, 8:136], flat[:, :1], flat[5:5]):
        check(m.quantize128(x, ROW | COLT, tile), x, tile, True)
        check(m.quantize128(x, ROW, tile), x, tile, True)


@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_values(tile, dtype):
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = torch.zeros(384, 384)
    x[0, :5] = torch.tensor([top, -top, 1.0, low, -low])
    x[130, :3] = torch.tensor([2.0 ** -101, -2.0 ** -108, 2.0 ** -120])  # below the floor of the scales
    x[1, 130:134] = torch.tensor([float("inf"), 1.0, -float("inf"), 0.0])
    x[140, 140:143] = torch.tensor([float("nan"), 2.0, float("inf")])
    x[300, 260] = 5e-39  # a subnormal
    x = x.to(dtype).cuda()
    check(mxq().quantize128(x, ROW | COLT, tile), x, tile, True)
    check(mxq().quantize128(x, ROW, tile), x, tile, True)


SIZES = [[5], [0, 1, 127, 128, 129, 0, 300, 2], [0, 0], [128, 256], [1] * 70, [0] * 100 + [3, 200] + [0] * 500 + [7]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axes", [COLT, ROW | COLT])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_grouped(case, axes, dtype):
    m, sizes = mxq(), SIZES[case]
    tail = 0 if case % 2 else 150  # rows of no group
    T, C = sum(sizes) + tail, 200
    x = spread((T, C), case, dtype)
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    P = sum(ref.up(n) for n in sizes)
    ldq = m.mxq_grouped128_cols_max(T, len(sizes))
    assert ldq >= P and ldq % 256 == 128
    out = {"q_row": torch.full((T, 256), GUARD, dtype=torch.uint8, device="cuda"), "s_row": torch.full((2, T), -1.0, device="cuda"),
           "q_colT": torch.full((C, ldq), GUARD, dtype=torch.uint8, device="cuda"), "s_colT": torch.full((ldq // 128, C), -1.0, device="cuda")}
    got = m.quantize128_grouped(x, ends, axes, out=out)
    assert got["ldq"] == ldq
    at = before = 0
    for n in sizes:
        if n:
            check_copy(got["q_colT"][:, before:before + ref.up(n)], got["s_colT"][before // 128:(before + ref.up(n)) // 128],
                       np.ascontiguousarray(wide(x[at:at + n]).T), 1, dtype == torch.bfloat16)
        at, before = at + n, before + ref.up(n)
    assert bool((got["q_colT"][:, P:] == GUARD).all()) and bool((got["s_colT"][P // 128:] == -1).all())
    if axes & ROW:
        check({k: got[k] for k in ("q_row", "s_row")}, x, 1, dtype == torch.bfloat16)


def test_grouped_narrow_and_malformed():
    """Blocks past ldq are dropped, and group ends out of order or out of range write nothing out of bounds."""
    m = mxq()
    x = spread((400, 130), 1, torch.bfloat16)
    for ends in ([150, 400], [400, 150], [-5, 10 ** 9], [300, 299], [2 ** 31 - 1, -2 ** 31]):
        whole = torch.full((131, 256), GUARD, dtype=torch.uint8, device="cuda")
        scales = torch.full((3, 130), -1.0, device="cuda")
        out = {"q_colT": whole[:130], "s_colT": scales[:2]}
        m.quantize128_grouped(x, torch.tensor(ends, dtype=torch.int32, device="cuda"), COLT, out=out)
        torch.cuda.synchronize()
        assert bool((whole[130] == GUARD).all()) and bool((scales[2] == -1).all())
    got = m.quantize128_grouped(x, torch.tensor([150, 400], dtype=torch.int32, device="cuda"), COLT, ldq=256)
    want, want_s = ref.quantize(np.ascontiguousarray(wide(x[:150]).T))
    assert np.array_equal(got["q_colT"].cpu().numpy(), want) and np.array_equal(got["s_colT"].cpu().numpy(), want_s)
