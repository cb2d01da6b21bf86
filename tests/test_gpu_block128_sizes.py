"""Block-128 quantisers and products at the sizes where another tile, wave layout or launch takes over, and past 32 bits."""
import numpy as np
import pytest
import torch

import block128_reference as ref
from gpu_util import mxq

pytestmark = pytest.mark.gpu
RAGGED_M, RAGGED_K = 0, 1


def operand(rows, K, seed, tile=1, lead=()):
    """Codes and scales drawn on the device: any finite code, scales over a few binades."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 127, (*lead, rows, K), generator=g, device="cuda", dtype=torch.uint8)
    codes |= torch.randint(0, 2, (*lead, rows, K), generator=g, device="cuda", dtype=torch.uint8) << 7
    return codes, torch.exp2(torch.rand((*lead, K // 128, -(-rows // tile)), generator=g, device="cuda") * 6 - 3)


def check(got, A, sA, B, sB):
    """Rows of a product, with the operands' rows that they are of."""
    want, f32, bf16 = ref.product_and_bounds(*(np.ascontiguousarray(t.cpu().numpy()) for t in (A, sA, B, sB)))
    err = np.abs(got.double().cpu().numpy() - want)
    bound = f32 if got.dtype == torch.float32 else bf16
    assert np.all(err <= bound), f"worst {np.max(err / np.maximum(bound, 1e-300)):.3g} of the bound"


def some(M, n=24):
    """Rows of M: the first and last, and where tiles of 64, 128 and 256 meet."""
    near = {0, M - 1, M // 2} | {k + d for k in (16, 64, 128, 256, M // 256 * 256, M // 128 * 128, M // 64 * 64) for d in (-1, 0)}
    return torch.tensor(sorted(i for i in near if 0 <= i < M)[:n], device="cuda")


# (M, N, K): 64 x 64 tiles, 128 x 128 with one workgroup a CU (K of 1 to 6 blocks: fewer and more than the stages), 128 x 128,
# 256 x 256, few rows with a wide N, few rows with a long K
DENSE = [(200, 1500, 384), (1100, 2000, 128), (1100, 2000, 256), (1100, 2000, 640), (1090, 2010, 768), (2100, 2200, 128), (2090, 2210, 384),
         (4000, 3400, 128), (3990, 3410, 384), (5, 33000, 256), (16, 32770, 128), (5, 40, 8448), (50, 8192, 256), (70, 8200, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("shape", DENSE)
def test_dense(shape, tile, dtype):
    M, N, K = shape
    A, sA = operand(M, K, 1)
    B, sB = operand(N, K, 2, tile)
    got = mxq().gemm128(A, sA, B, sB, dtype=dtype)
    rows, cols = some(M), some(N)
    if tile == 1:
        check(got[:, cols], A, sA, B[cols], sB[:, cols])
    check(got[rows], A[rows], sA[:, rows], B, sB)


def sizes_of(T, G, seed):
    """G groups of uneven sizes with sum T, some empty."""
    cuts = np.sort(np.random.default_rng(seed).integers(0, T + 1, G - 1))
    cuts[:len(cuts) // 4] = 0
    return np.diff(np.concatenate([[0], cuts, [T]]))


# (T, G, N, K): tiles of each shape, few rows with many and few workgroups (rows a group up to 16, 32, 64), 1024 groups
MOE = [(500, 3, 500, 256), (1000, 6, 2000, 384), (1300, 6, 2000, 384), (3000, 5, 4200, 256), (3000, 7, 2200, 128), (36, 9, 4100, 128), (60, 9, 4100, 256), (140, 9, 4100, 128),
       (36, 9, 300, 128), (60, 9, 300, 1152), (140, 9, 300, 256), (2000, 1024, 130, 128), (60000, 1024, 64, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", MOE)
def test_ragged_m(case, dtype):
    T, G, N, K = case
    ragged_m(sizes_of(T, G, 5), N, K, dtype)


# few rows a group on average, all or most of them in one or two
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [[0] * 30 + [64] + [0] * 9, [0, 65] + [0] * 38, [0] * 39 + [150], [129] + [1] * 37 + [0, 64], [0, 300, 1, 128, 0] * 8,
                                   [64] * 20 + [65] * 20, [1] * 500 + [500] + [0] * 499])
def test_few_rows_in_uneven_groups(sizes, dtype):
    ragged_m(np.array(sizes), 200, 256, dtype)


def ragged_m(sizes, N, K, dtype):
    T, G = int(sizes.sum()), len(sizes)
    A, sA = operand(T + 9, K, 3)
    B, sB = operand(N, K, 4, 128, (G,))
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    C = torch.full((T + 9, N), 7.0, dtype=dtype, device="cuda")
    mxq().mxq_grouped_gemm128(RAGGED_M, A, sA, B, sB, C, ends)
    assert bool((C[T:] == 7).all())
    at = 0
    for g, m in enumerate(sizes):
        if m and (G < 64 or m > 1 and g % 97 == 0 or m > 300 or g == G - 1):
            rows = at + some(int(m))
            check(C[rows], A[rows], sA[:, rows], B[g], sB[g])
        at += m


# (sizes, M, N): tiles of each shape, 37 groups of few tiles, 1024 of them
WEIGHTS = [([130, 0, 5, 300], 200, 300), ([1, 129, 0, 700], 700, 500), ([1, 129, 0, 700], 1100, 500), ([300, 0, 140], 2100, 1200), ([7 * i % 190 for i in range(37)], 200, 340),
           ([0, 257] * 512, 70, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_ragged_k(case, dtype):
    sizes, M, N = WEIGHTS[case]
    starts = np.concatenate([[0], np.cumsum([ref.up(m) for m in sizes])])
    ldq = int(starts[-1]) + 128
    A, sA = operand(M, ldq, 6)
    B, sB = operand(N, ldq, 7)
    for q, s in ((A, sA), (B, sB)):  # past the last group: NaN
        q[:, starts[-1]:], s[starts[-1] // 128:] = 0x7F, float("nan")
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    got = mxq().grouped_gemm128(RAGGED_K, A, sA, B, sB, ends, dtype=dtype)
    rows = some(M)
    for g, m in enumerate(sizes):
        if m == 0:
            assert bool((got[g] == 0).all())
        elif len(sizes) < 64 or g % 301 == 0 or g == len(sizes) - 1:
            k, b = slice(starts[g], starts[g + 1]), slice(starts[g] // 128, starts[g + 1] // 128)
            check(got[g][rows], A[rows][:, k], sA[b][:, rows], B[:, k], sB[b])


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 2 ** 30:
        pytest.skip("needs more device memory")


def test_output_past_32_bits():
    room(12)
    M, N, K = 70000, 33000, 128
    A, sA = operand(M, K, 1)
    B, sB = operand(N, K, 2, 128)
    got = mxq().gemm128(A, sA, B, sB)
    rows = torch.tensor([0, 32539, 65075, 65076, M - 1], device="cuda")  # around 2^30 and 2^31 elements
    check(got[rows], A[rows], sA[:, rows], B, sB)


@pytest.mark.parametrize("T", [70, 40000])
def test_weights_past_32_bits(T):
    room(16)
    G, N, K = 40, 8000, 7168
    B, sB = operand(N, K, 2, 128, (G,))
    A, sA = operand(T, K, 1)
    ends = torch.full((G,), T, dtype=torch.int32, device="cuda")  # all rows in the last but one group, or spread
    ends[:-2] = 0
    got = mxq().grouped_gemm128(RAGGED_M, A, sA, B, sB, ends)
    rows = torch.tensor([0, 1, T - 1], device="cuda")
    check(got[rows], A[rows], sA[:, rows], B[G - 2], sB[G - 2])


def test_quantiser_past_32_bits():
    room(24)
    R, C = 300000, 8000
    m = mxq()
    x = torch.randn(1000, C, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16().repeat(R // 1000, 1)
    for tile in (1, 128):
        got = m.quantize128(x, 3, tile)
        if tile == 1:
            part = m.quantize128(x[-1000:], 1)
            assert torch.equal(got["q_row"][-1000:], part["q_row"]) and torch.equal(got["s_row"][:, -1000:], part["s_row"])
        last = R // 128 * 128 - 128 * 3
        part = m.quantize128(x[last:], 3, tile)
        assert torch.equal(got["q_colT"][:, last:], part["q_colT"]) and torch.equal(got["s_colT"][last // 128:], part["s_colT"])
        if tile == 128:
            assert torch.equal(got["q_row"][last:], part["q_row"]) and torch.equal(got["s_row"][:, last // 128:], part["s_row"])
        del got


@pytest.mark.parametrize("axes,R", [(1, 2 ** 28 + 100), (2, 2 ** 31 - 1)])
def test_more_workgroups_than_a_launch_has(axes, R):
    room(64)
    x = torch.ones(R, 1, dtype=torch.bfloat16, device="cuda")
    x[-70:] = -2.0
    got = mxq().quantize128(x, axes)
    name = "row" if axes == 1 else "colT"
    codes, scales = got["q_" + name], got["s_" + name].view(-1)
    codes = codes[:, 0] if axes == 1 else codes[0, :R]
    assert bool((codes[-70:] == 0xFE).all())
    if axes == 1:
        assert all(bool((c == 0x7E).all()) for c in codes[:-70].split(2 ** 27))
        want = torch.tensor([1.0, 2.0], device="cuda") / 448
        assert bool((scales[-70:] == want[1]).all()) and bool((scales[:-70] == want[0]).all())
    else:  # the last block has 127 columns, 57 of 1 and 70 of -2
        assert all(bool((c == 0x7E).all()) for c in codes[:-127].split(2 ** 29)) and bool((codes[-127:-70] == 0x76).all())
        want = torch.tensor([1.0, 2.0], device="cuda") / 448
        assert scales[-1] == want[1] and bool((scales[:-1] == want[0]).all())
