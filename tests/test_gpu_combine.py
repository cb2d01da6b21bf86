"""Combine, its gradient and the dispatch against 64-bit references.

A sum of K products in fp32 is off by at most (K + 1) half steps of sum |w y|, a dot product over H whose
longest chain of additions is H / 64 + 16 by that many of sum |d y|; a result rounded to bf16 by half a
step more."""
import numpy as np
import pytest
import torch

import moe_reference as ref
from gpu_util import host, mxq

pytestmark = pytest.mark.gpu

TYPES = (torch.float32, torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def case(T, K, H, ydt, odt, seed, dropped=0.0, extra=3):
    g = torch.Generator().manual_seed(seed)
    rows = T * K + extra
    slot = torch.randperm(rows, generator=g)[:T * K].to(torch.int32).view(T, K)
    if dropped and T:
        slot[torch.rand(T, K, generator=g) < dropped] = -1
        slot[T // 2] = -1
        slot[0, 0] = rows
        slot[-1, -1] = 2 ** 31 - 1
        slot[T // 3, 0] = -2 ** 31
    y = torch.randn(rows, H, generator=g).to(ydt)
    w = torch.randn(T, K, generator=g)
    d = torch.randn(T, H, generator=g).to(odt)
    return rows, slot.cuda(), y.cuda(), w.cuda(), d.cuda()


def used(slot, rows):
    s = host(slot).astype(np.int64)
    ok = (s >= 0) & (s < rows)
    return np.where(ok, s, 0), ok


def check_combine(y, slot, w, odt, out=None):
    m = mxq()
    if out is None:
        out = m.combine(y, slot, w, dtype=odt)
    else:
        m.mxq_combine(y, slot, w, out)
    s, ok = used(slot, y.shape[0])
    wt = np.where(ok, 1.0 if w is None else f64(w), 0.0)
    rows = f64(y)[s] if y.shape[0] else np.zeros(s.shape + (y.shape[1],))
    want = (wt[:, :, None] * rows).sum(1)
    size = (np.abs(wt)[:, :, None] * np.abs(rows)).sum(1)
    tol = (slot.shape[1] + 1) * ref.U32 * size + (ref.UBF16 * (np.abs(want) + ref.U32 * 40 * size) if odt == torch.bfloat16 else 0)
    assert np.all(np.abs(f64(out) - want) <= tol)
    if slot.numel():
        assert not f64(out)[~ok.any(1)].any()  # a token without experts


def check_backward(d, slot, rows, w, y, gdt):
    m = mxq()
    s, ok = used(slot, rows)
    T, K = s.shape
    H = d.shape[1]
    dy = torch.full((rows, H), 7.0, dtype=gdt, device="cuda")
    dw = None if y is None else torch.full((T, K), 7.0, device="cuda")
    m.mxq_combine_backward(d, slot, rows, dy, dw, w, y)
    got = f64(dy)
    want = np.full((rows, H), 7.0)
    for t, k in zip(*np.nonzero(ok)):
        want[s[t, k]] = f64(d)[t] * (1.0 if w is None else f64(w)[t, k])
    half = ref.U32 if gdt == torch.float32 else ref.UBF16 * (1 + 2.0 ** -14)
    assert np.all(np.abs(got - want) <= half * np.abs(want))
    assert np.array_equal(got[np.setdiff1d(np.arange(rows), s[ok])], np.full((rows - ok.sum(), H), 7.0))  # not written
    if dw is not None:
        prod = f64(y)[s] * f64(d)[:, None, :] if rows else np.zeros((T, K, H))
        want = np.where(ok, prod.sum(2), 0.0)
        tol = (H / 64 + 16) * ref.U32 * np.where(ok, np.abs(prod).sum(2), 0.0)
        assert np.all(np.abs(f64(dw) - want) <= tol)
        dw2 = torch.empty_like(dw)
        m.mxq_combine_backward(d, slot, rows, None, dw2, w, y)
        assert torch.equal(dw, dw2)


SIZES = [(0, 2, 8), (1, 1, 1), (1, 8, 7), (3, 2, 64), (5, 3, 129), (7, 8, 1000), (2, 32, 1024), (33, 8, 2048), (16, 6, 4095),
         (9, 4, 4104), (3, 8, 7168), (2, 2, 20000), (70, 1, 256), (6, 5, 520), (3, 7, 264), (4, 9, 1030), (2, 11, 100),
         (2, 17, 65)]


@pytest.mark.parametrize("ydt", TYPES)
@pytest.mark.parametrize("odt", TYPES)
@pytest.mark.parametrize("T,K,H", SIZES)
def test_combine(T, K, H, ydt, odt):
    for dropped in (0.0, 0.4):
        rows, slot, y, w, _ = case(T, K, H, ydt, odt, T + H, dropped)
        check_combine(y, slot, w, odt)
        check_combine(y, slot, None, odt)


@pytest.mark.parametrize("ydt", TYPES)
@pytest.mark.parametrize("odt", TYPES)
@pytest.mark.parametrize("T,K,H", SIZES)
def test_combine_backward(T, K, H, ydt, odt):
    for dropped in (0.0, 0.4):
        rows, slot, y, w, d = case(T, K, H, ydt, odt, T + H, dropped)
        for gdt in TYPES:
            check_backward(d, slot, rows, w, y, gdt)
            check_backward(d, slot, rows, None, y, gdt)
            check_backward(d, slot, rows, w, None, gdt)
            check_backward(d, slot, rows, None, None, gdt)


def test_dispatch_is_a_gather():
    m = mxq()
    for dt in TYPES:
        x = torch.randn(37, 200, device="cuda").to(dt)
        x[3, 5], x[4, 6], x[5, 7] = float("nan"), float("inf"), -0.0
        r = m.route(torch.randn(37, 16, device="cuda"), 4)
        rows = m.dispatch(x, r["slot"], 37 * 4)
        want = x[r["row_token"].long()]
        bits = torch.int32 if dt == torch.float32 else torch.int16
        assert torch.equal(rows.view(bits), want.view(bits))


def test_combine_passes_infinities_and_nan():
    """Values of rows that a slot names go through; those of rows that none names do not."""
    y = torch.ones(4, 16, device="cuda")
    y[0, 1], y[1, 2], y[3] = float("inf"), float("nan"), float("nan")
    slot = torch.tensor([[0, 1], [2, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    out = mxq().combine(y, slot, torch.ones(3, 2, device="cuda"), dtype=torch.float32)
    assert bool(torch.isinf(out[0, 1])) and bool(torch.isnan(out[0, 2])) and bool((out[1] == 1).all()) and bool((out[2] == 0).all())


def test_no_rows_at_all():
    m = mxq()
    slot = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(4, 3, device="cuda")
    y = torch.empty(0, 40, device="cuda")
    assert not bool(m.combine(y, slot, w, dtype=torch.float32).any())
    dy, dw = m.combine_backward(torch.ones(4, 40, device="cuda"), slot, 0, w, y)
    assert dy.shape == (0, 40) and not bool(dw.any())


@pytest.mark.parametrize("lo,hi,H", [(0, 512, 512), (1, 301, 400), (8, 264, 264), (3, 4, 9)])
def test_strides_and_alignment(lo, hi, H):
    """Rows that are parts of wider ones, at offsets that break 16-byte alignment."""
    for ydt in TYPES:
        for odt in TYPES:
            rows, slot, y, w, d = case(11, 4, H, ydt, odt, H, 0.2)
            wide = torch.full((11, H + 5), 7.0, dtype=odt, device="cuda")
            check_combine(y[:, lo:hi], slot, w, odt, out=wide[:, lo:hi])
            assert bool((wide[:, hi:] == 7).all()) and bool((wide[:, :lo] == 7).all())
            m = mxq()
            a = m.combine_backward(d[:, lo:hi], slot, rows, w, y[:, lo:hi])
            b = m.combine_backward(d[:, lo:hi].contiguous(), slot, rows, w, y[:, lo:hi].contiguous())
            s, ok = used(slot, rows)
            assert torch.equal(a[0][s[ok]], b[0][s[ok]])
            tol = (hi / 64 + 16) * 2 * ref.U32 * np.where(ok, np.abs(f64(y)[s][:, :, lo:hi] * f64(d)[:, None, lo:hi]).sum(2), 0)
            assert np.all(np.abs(f64(a[1]) - f64(b[1])) <= tol)


def test_gradient_against_differences():
    """The combine is linear in y and in w, so one difference of any size is exact up to rounding: fp32 values of
    two results, off by at most (K + 1) half steps of sum |w y| each."""
    m = mxq()
    rows, slot, y, w, d = case(3, 4, 33, torch.float32, torch.float32, 5)
    dy, dw = m.combine_backward(d, slot, rows, w, y)
    base = m.combine(y, slot, w, dtype=torch.float32)
    size = float((w.abs()[:, :, None] * y[slot.long()].abs()).sum(1).max()) + 10
    for t in range(3):
        for k in range(4):
            w2 = w.clone()
            w2[t, k] += 1.0
            diff = ((m.combine(y, slot, w2, dtype=torch.float32) - base).double() * d.double()).sum()
            assert abs(float(diff) - float(dw[t, k])) <= 33 * 5 * 12 * ref.U32 * size
            y2 = y.clone()
            y2[slot[t, k].long(), 7] += 1.0
            diff = ((m.combine(y2, slot, w, dtype=torch.float32) - base).double() * d.double()).sum()
            assert abs(float(diff) - float(dy[slot[t, k].long(), 7])) <= 33 * 5 * 12 * ref.U32 * size


def test_rows_past_32_bits():
    """Rows whose elements lie past 2^32 of the first."""
    m = mxq()
    H, rows = 8192, (1 << 19) + 40
    y = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([[rows - 1, 5], [rows - 17, 1 << 19]], dtype=torch.int32, device="cuda")
    small = torch.randn(4, H, device="cuda").to(torch.bfloat16)
    y[slot.view(-1).long()] = small
    w = torch.randn(2, 2, device="cuda")
    near = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    assert torch.equal(m.combine(y, slot, w), m.combine(small, near, w))
    d = torch.randn(2, H, device="cuda").to(torch.bfloat16)
    dy, dw = m.combine_backward(d, near, 4, w, small)
    _, dw2 = m.combine_backward(d, slot, rows, w, y)
    assert torch.equal(dw, dw2)
    m.mxq_combine_backward(d, slot, rows, y, None, w)
    assert torch.equal(y[slot.view(-1).long()], dy)


def test_on_another_stream():
    m = mxq()
    rows, slot, y, w, d = case(50, 4, 512, torch.float32, torch.bfloat16, 6)
    want, grads = m.combine(y, slot, w), m.combine_backward(d, slot, rows, w, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got, g2 = m.combine(y, slot, w), m.combine_backward(d, slot, rows, w, y)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(grads[1], g2[1])
    assert torch.equal(grads[0][slot.long()], g2[0][slot.long()])


def test_helpers_refuse_other_types():
    m = mxq()
    y, slot = torch.zeros(4, 8, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    with pytest.raises(TypeError, match="dtype must be"):
        m.combine(y, slot, dtype=torch.float16)
    with pytest.raises(TypeError, match="dtype must be"):
        m.dispatch(y[:2], slot, 4, dtype=torch.float64)


@pytest.mark.parametrize("ydt", TYPES)
@pytest.mark.parametrize("odt", TYPES)
@pytest.mark.parametrize("T,K,H", [(257, 3, 2056), (257, 8, 4096), (257, 2, 4104), (300, 5, 7168)])
def test_workgroups_of_more_than_four_waves(T, K, H, ydt, odt):
    """From 256 tokens on, rows of more than 2048 columns take 5 to 8 waves a workgroup."""
    rows, slot, y, w, d = case(T, K, H, ydt, odt, T + H, 0.2)
    check_combine(y, slot, w, odt)
    check_combine(y, slot, None, odt)
    for gdt in TYPES:
        check_backward(d, slot, rows, w, y, gdt)
    check_backward(d, slot, rows, None, None, odt)
