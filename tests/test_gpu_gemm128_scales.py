"""Block-128 products of scales far apart, to the ends of fp32's range."""
import numpy as np
import pytest
import torch

from gpu_util import mxq

pytestmark = pytest.mark.gpu

ONE = 0x38  # E4M3's 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b_tile", [1, 128])
@pytest.mark.parametrize("M", [5, 40, 300])
def test_powers_of_two(M, b_tile, dtype):
    """One product of 1 x 1 a block: C = sA sB of the first block plus 0 of the second, exactly; the products of scales run
    from the least normal number to 2^126."""
    N, K = 300, 256
    A, B = torch.zeros(M, K, dtype=torch.uint8), torch.zeros(N, K, dtype=torch.uint8)
    A[:, 17] = ONE
    B[:, 17] = ONE
    r = np.random.default_rng(M + b_tile)
    ea, eb = r.integers(-63, 64, (2, M)), r.integers(-63, 64, (2, N if b_tile == 1 else 3))
    sA, sB = (torch.from_numpy(np.exp2(e.astype(np.float64)).astype(np.float32)).cuda() for e in (ea, eb))
    C = mxq().gemm128(A.cuda(), sA, B.cuda(), sB, dtype=dtype)
    want = np.exp2((ea[0][:, None] + np.repeat(eb[0], b_tile)[None, :N]).astype(np.float64))
    assert np.array_equal(C.double().cpu().numpy(), want)


@pytest.mark.parametrize("M", [5, 300])
def test_a_small_scale_against_a_large_one(M):
    """Rows whose scales are 2^100 against columns whose scales are 2^-100, and the other way round."""
    N, K = 130, 128
    A, B = torch.full((M, K), ONE, dtype=torch.uint8).cuda(), torch.full((N, K), ONE, dtype=torch.uint8).cuda()
    for e in (100, -100):
        for b_tile, n in ((1, N), (128, 2)):
            C = mxq().gemm128(A, torch.full((1, M), 2.0 ** e, device="cuda"), B, torch.full((1, n), 2.0 ** -e, device="cuda"), dtype=torch.float32)
            assert bool((C == 128).all()), (e, b_tile)
