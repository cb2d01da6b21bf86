"""FP8 with one scale for every block of 128, in 64 bits on the host: the quantiser, operands' values and the products."""
import numpy as np

BLOCK = 128
FLOOR = 2.0 ** -100


def up(n):
    return -(-n // BLOCK) * BLOCK


def e4m3_table():
    """Values of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


TABLE = e4m3_table()


def step_of(y):
    """Distance of the E4M3 values around y: 2^(exponent - 3), no smaller than 2^-9."""
    _, e = np.frexp(y)
    return np.exp2(np.maximum(e - 1, -6) - 3.0)


def nearest_code(y):
    """Codes nearest to y (|y| <= 448), ties to even; a zero keeps its sign, NaN is 0x7F."""
    step = step_of(np.where(np.isfinite(y), y, 0.0))
    v = np.abs(np.rint(np.where(np.isfinite(y), y, 0.0) / step) * step)
    code = np.searchsorted(TABLE[:127], v).astype(np.uint8)  # (v is one of the values)
    assert np.array_equal(TABLE[code], v)
    return np.where(np.isfinite(y), code | (np.signbit(y) << 7), 0x7F).astype(np.uint8)


def blocks_amax(x, tile):
    """amax [ceil(R / tile)][ceil(C / 128)] of a 64-bit matrix; NaN where a block has one."""
    R, C = x.shape
    p = np.zeros((-(-R // tile) * tile, up(C)))
    p[:R, :C] = np.abs(x)
    m = p.reshape(p.shape[0] // tile, tile, p.shape[1] // BLOCK, BLOCK).max(axis=(1, 3))
    return np.where(np.isnan(m), m, np.maximum(m, FLOOR))


def quotients(x, tile):
    """448 x / amax [R][ceil128(C)], zero past C."""
    R, C = x.shape
    each = np.repeat(np.repeat(blocks_amax(x, tile), tile, 0)[:R], BLOCK, 1)
    p = np.zeros((R, up(C)))
    p[:, :C] = x
    with np.errstate(invalid="ignore"):
        return p * 448.0 / each


def quantize(x, tile=1):
    """Row copy of x (64-bit values): codes [R][ceil128(C)], scales fp32 [C / 128][R / tile]."""
    with np.errstate(over="ignore"):
        scales = (blocks_amax(x, tile).astype(np.float32) / np.float32(448)).T
    return nearest_code(quotients(x, tile)), np.ascontiguousarray(scales)


def quantize_grouped(x, sizes, ldq=None):
    """colT copy of x [T][C] with blocks restarting at each group: codes [C][P], scales [P / 128][C]."""
    codes, scales, at = [np.zeros((x.shape[1], 0), np.uint8)], [np.zeros((0, x.shape[1]), np.float32)], 0
    for m in sizes:
        if m:
            q, s = quantize(np.ascontiguousarray(x[at:at + m].T))
            codes.append(q)
            scales.append(s)
        at += m
    return np.concatenate(codes, 1), np.concatenate(scales, 0)


def values(codes, scales):
    """64-bit values of an operand [rows][K] with scales [K / 128][rows] or [K / 128][ceil(rows / 128)]."""
    rows = codes.shape[0]
    s = scales.astype(np.float64).T
    if s.shape[0] != rows:
        s = np.repeat(s, BLOCK, 0)[:rows]
    return TABLE[codes] * np.repeat(s, BLOCK, 1)


def product_and_bounds(A, sA, B, sB):
    """fp64 A B^T of two operands, and how far an fp32 and a bf16 output may be from it.

    fp32: exact products, 128 of them and then the blocks added with a relative error of at most 2^-23 each (an addition
    that cuts), and the scales' product, its multiplication and the sum rounded.  bf16: a group of eight products of
    consecutive k keeps 13 bits below its largest, so it is off by at most 8 * 2^-13 of that, and the result is rounded
    to nearest, by half a step."""
    a, b = values(A, sA), values(B, sB)
    ref = a @ b.T
    total = np.abs(a) @ np.abs(b).T
    K = A.shape[1]
    f32 = (BLOCK + K // BLOCK + 4) * 2.0 ** -23 * total
    ga, gb = np.abs(a).reshape(len(a), -1, 8), np.abs(b).reshape(len(b), -1, 8)
    groups = np.zeros_like(ref)
    for j in range(K // 8):
        groups += (ga[:, None, j] * gb[None, :, j]).max(-1)
    near = f32 + 8 * 2.0 ** -13 * groups
    return ref, f32, near + 2.0 ** -8 * (np.abs(ref) + near)
