"""Products of FP8 operands with a scale for each block of 128 against the 64-bit product of their values."""
import numpy as np
import pytest
import torch

import block128_reference as ref
from gpu_util import mxq

pytestmark = pytest.mark.gpu
RAGGED_M, RAGGED_K = 0, 1


def operand(rows, K, seed, tile=1, odd=0.3):
    """Codes and scales as a quantiser leaves them: N(0, 1) values, columns of very different size, zeros past K."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, K)) * np.exp2(r.integers(-6, 7, (rows, 1))) * np.where(r.random(K) < 0.05, 20.0, 1.0)
    return ref.quantize(x, tile)


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def check(got, A, sA, B, sB):
    want, f32, bf16 = ref.product_and_bounds(A, sA, B, sB)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = f32 if got.dtype == torch.float32 else bf16
    assert np.all(err <= bound), f"worst {np.max(err / np.maximum(bound, 1e-300)):.3g} of the bound"


SHAPES = [(1, 1, 128), (7, 300, 300), (16, 128, 1024), (17, 129, 257), (33, 64, 130), (64, 200, 512), (65, 130, 384), (128, 128, 128),
          (130, 260, 640), (257, 511, 256), (200, 40, 2048)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_dense(shape, tile, dtype):
    M, N, K = shape
    A, sA = operand(M, K, M + N)
    B, sB = operand(N, K, K, tile)
    got = mxq().gemm128(*dev(A, sA, B, sB), dtype=dtype)
    assert got.shape == (M, N) and got.dtype == dtype
    check(got, A, sA, B, sB)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [5, 70, 140])
def test_output_rows_apart(M, dtype):
    """A wider C: nothing is written past N."""
    A, sA = operand(M, 256, 1)
    B, sB = operand(99, 256, 2, 128)
    for at in (0, 1, 8):
        C = torch.full((M, 140), 7.0, dtype=dtype, device="cuda")
        mxq().mxq_gemm128(*dev(A, sA, B, sB), C[:, at:at + 99])
        check(C[:, at:at + 99], A, sA, B, sB)
        assert bool((C[:, :at] == 7).all()) and bool((C[:, at + 99:] == 7).all())


def groups(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


SIZES = [[3], [0, 1, 16, 17, 0, 40], [130, 0, 5], [1] * 9, [0, 0], [64, 65, 300], [0] * 70 + [2, 33] + [0] * 5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(130, 256), (64, 128), (300, 640)])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_ragged_m(case, N, K, dtype):
    sizes = SIZES[case]
    G, tail = len(sizes), case % 2 * 3
    T = sum(sizes) + tail
    A, sA = operand(T, K, 7) if T else (np.zeros((0, K), np.uint8), np.zeros((K // 128, 0), np.float32))
    pairs = [operand(N, K, 100 + g, 128) for g in range(G)]
    B, sB = np.stack([p[0] for p in pairs]), np.stack([p[1] for p in pairs])
    C = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    mxq().mxq_grouped_gemm128(RAGGED_M, *dev(A, sA, B, sB), C, groups(sizes))
    at = 0
    for g, m in enumerate(sizes):
        if m:
            check(C[at:at + m], A[at:at + m], np.ascontiguousarray(sA[:, at:at + m]), B[g], sB[g])
        at += m
    assert bool((C[at:] == 7).all())


K_SIZES = [[3], [0, 1, 127, 128, 129, 0, 300], [0, 0], [256, 128], [1] * 70]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(130, 70), (16, 300), (1, 1)])
@pytest.mark.parametrize("case", range(len(K_SIZES)))
def test_ragged_k(case, M, N, dtype):
    sizes = K_SIZES[case]
    r = np.random.default_rng(case)
    T, P = sum(sizes), sum(ref.up(m) for m in sizes)
    ldq = max(128, P) + 128 * (case % 2)
    ops = []
    for rows in (M, N):
        codes, scales = ref.quantize_grouped(r.standard_normal((T, rows)) * np.exp2(r.integers(-6, 7, (T, 1))), sizes)
        q, s = np.full((rows, ldq), 0x7F, np.uint8), np.full((ldq // 128, rows), np.nan, np.float32)  # past the last group: NaN
        q[:, :P], s[:P // 128] = codes, scales
        ops += [q, s]
    got = mxq().grouped_gemm128(RAGGED_K, *dev(*ops), groups(sizes), dtype=dtype)
    assert got.shape == (len(sizes), M, N)
    before = 0
    for g, m in enumerate(sizes):
        if m == 0:
            assert bool((got[g] == 0).all())
            continue
        cols, blocks = slice(before, before + ref.up(m)), slice(before // 128, (before + ref.up(m)) // 128)
        check(got[g], *(np.ascontiguousarray(v) for v in (ops[0][:, cols], ops[1][blocks], ops[2][:, cols], ops[3][blocks])))
        before += ref.up(m)


def test_malformed_group_ends_stay_in_bounds():
    m = mxq()
    A, sA = operand(200, 256, 1)
    pairs = [operand(130, 256, g, 128) for g in range(2)]
    B, sB = np.stack([p[0] for p in pairs]), np.stack([p[1] for p in pairs])
    for ends in ([150, 100], [-5, 10 ** 9], [2 ** 31 - 1, -2 ** 31]):
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        whole = torch.full((201, 130), 7.0, device="cuda")
        m.mxq_grouped_gemm128(RAGGED_M, *dev(A, sA, B, sB), whole[:200], e)
        k = torch.full((3, 200, 200), 7.0, device="cuda")
        m.mxq_grouped_gemm128(RAGGED_K, *dev(A, sA, A, sA), k[:2], e)
        torch.cuda.synchronize()
        assert bool((whole[200] == 7).all()) and bool((k[2] == 7).all())


def test_special_values():
    """NaN and infinite scales and codes reach their rows and columns alone."""
    m = mxq()
    A, sA = operand(40, 256, 1)
    B, sB = operand(130, 256, 2)
    A[3, 17] = 0x7F
    sA[1, 5] = np.inf
    sB[0, 9] = np.nan
    for dtype in (torch.bfloat16, torch.float32):
        C = m.gemm128(*dev(A, sA, B, sB), dtype=dtype).cpu()
        bad = ~torch.isfinite(C)
        want = torch.zeros(40, 130, dtype=torch.bool)
        want[[3, 5]] = True
        want[:, 9] = True
        assert torch.equal(bad, want)
