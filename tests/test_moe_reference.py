"""What pins the 64-bit references of the router, combine and AdamW tests: torch's types, autograd and differences."""
import numpy as np
import pytest
import torch

import moe_reference as ref


def test_e4m3_table_is_torchs():
    assert np.array_equal(ref.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


def test_encode_rounds_without_bias_between_neighbours():
    """Over all u, the mean of the rounded values is the value: (number of u) / 65536 of a step at most off."""
    x = np.array([448.0, 0.3, 17.3, 1e-3, 2.0 ** -9, 5e-4, 0.0, -0.7])
    u = (np.arange(65536) + 0.5) / 65536
    got = np.stack([ref.decode(*ref.encode(x, np.full(len(x), v))[:2]) for v in u[::64]])
    step = np.where(np.abs(x) < 2.0 ** -6, 2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3))
    assert np.all(np.abs(got.mean(0) - x) <= step / 1024)
    lo = np.abs(got) <= np.abs(x) + step
    assert lo.all()


@pytest.mark.parametrize("positive", [False, True])
def test_encode_scales(positive):
    """The scale is the smallest power of two that keeps the block at or below 448."""
    for amax in (448.0, 449.0, 1.75, 1.7500001, 3e-38, 1e30, 2.0 ** -100):
        x = np.zeros(40)
        x[7], x[35] = amax, amax / 3
        codes, scales, _, _ = ref.encode(x, np.full(40, 1e-3), positive)
        for b, top in ((0, amax), (1, amax / 3)):
            s = 2.0 ** (int(scales[b]) - 127)
            assert top / s <= 448 and (scales[b] == 1 or top / (s / 2) > 448)


def test_positive_values_do_not_vanish():
    x = np.array([1.0] + [1e-9] * 31)
    codes, scales, _, _ = ref.encode(x, np.full(32, 1e-4), True)
    assert np.all(codes >= 1) and not ref.encode(x, np.full(32, 1e-4))[0][1:].any()


def test_random_bits_are_uniform_and_uncorrelated():
    n = 1 << 18
    prev = None
    for step, tensor in ((1, 0), (2, 0), (1, 1), (100000, 39)):
        for u in ref.uniforms(99, step, tensor, n):
            assert abs(u.mean() - 0.5) < 5 / np.sqrt(12 * n)
            for part in (u[::2], u[1::2]):
                c = np.bincount((part * 64).astype(int), minlength=64)
                assert ((c - n / 128) ** 2 / (n / 128)).sum() < 63 + 6 * np.sqrt(2 * 63)
            for lag in (1, 2, 32):
                assert abs(np.corrcoef(u[:-lag], u[lag:])[0, 1]) < 6 / np.sqrt(n)
            if prev is not None:
                assert abs(np.corrcoef(u, prev)[0, 1]) < 6 / np.sqrt(n)
            prev = u


def test_uniforms_of_a_later_range():
    a, b = ref.uniforms(3, 4, 5, 1000), ref.uniforms(3, 4, 5, 900, 100)
    assert np.array_equal(a[0][100:], b[0]) and np.array_equal(a[1][100:], b[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward_is_autograds(score, renormalise):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 12, generator=g, dtype=torch.float64, requires_grad=True)
    idx, w = ref.route(x.detach().numpy(), 3, score, renormalise=renormalise, scale=2.0)
    dw = torch.randn(5, 3, generator=g, dtype=torch.float64)
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    wt = s.gather(1, torch.from_numpy(idx).long())
    if renormalise:
        wt = wt / wt.sum(1, keepdim=True)
    wt = 2.0 * wt
    assert np.allclose(wt.detach().numpy(), w, rtol=1e-14)
    (wt * dw).sum().backward()
    got = ref.route_backward(x.detach().numpy(), idx, dw.numpy(), score, renormalise, 2.0)
    assert np.allclose(got, x.grad.numpy(), rtol=1e-12, atol=1e-14)


def test_route_selection():
    """A case written out by hand: two groups, the first has the best pair, a mask and a tie."""
    l = np.array([[2.0, 1.0, 0.0, -np.inf, 3.0, -5.0, -5.0, -5.0]])
    assert ref.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=2)[0].tolist() == [[0, 1]]
    assert ref.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=1)[0].tolist() == [[4, 5]]
    assert ref.route(l, 5, "softmax", n_group=2, topk_group=1, group_top=2)[0].tolist() == [[4, 5, 6, 7, -1]]  # e^3 > e^2 + e
    assert ref.route(l, 5, "sigmoid", n_group=2, topk_group=1, group_top=2)[0].tolist() == [[0, 1, 2, -1, -1]]
    b = np.array([0, 0, 5.0, 9.0, 0, 0, 0, 0])
    assert ref.route(l, 2, "sigmoid", bias=b)[0].tolist() == [[2, 4]]


def test_expert_order_is_a_stable_sort():
    idx = np.array([[2, 0], [0, -1], [2, 1], [7, 0]], np.int32)
    ends, token, slot = ref.expert_order(idx, 3)
    assert ends.tolist() == [3, 4, 6] and token.tolist() == [0, 1, 3, 2, 0, 2, -1, -1]
    assert slot.tolist() == [[4, 0], [1, -1], [5, 3], [-1, 2]]


def test_adamw_is_torchs():
    g = torch.Generator().manual_seed(1)
    p = torch.randn(50, generator=g, dtype=torch.float64)
    gr = torch.randn(50, generator=g, dtype=torch.float64)
    q = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([q], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m = v = np.zeros(50)
    x = p.numpy()
    for t in (1, 2, 3):
        q.grad = gr * t
        opt.step()
        x, m, v, _, _, _ = ref.adamw(x, gr.numpy() * t, m, v, 0.01, (0.8, 0.95), 1e-6, 0.1, t, 1.0)
        assert np.allclose(x, q.detach().numpy(), rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_references_of_many_rows(score, renormalise):
    """The vectorised references are those of one row at a time."""
    rng = np.random.default_rng(3)
    l = rng.standard_normal((40, 24))
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[7] = -np.inf
    l[8] = np.round(l[8])
    for bias in (None, rng.standard_normal(24) * 0.2):
        for groups in ({}, dict(n_group=4, topk_group=2, group_top=2), dict(n_group=6, topk_group=1, group_top=1)):
            kw = dict(score=score, bias=bias, renormalise=renormalise, scale=1.5, **groups)
            (i, w), (ri, rw) = ref.route(l, 5, **kw), ref.route_rows(l, 5, **kw)
            assert np.array_equal(i, ri) and np.allclose(w, rw, rtol=1e-14, atol=0)
    idx = ref.route(l, 5, score)[0]
    idx[3, 2], idx[4, 0] = 24, -(2 ** 31)
    dw = rng.standard_normal(idx.shape)
    a, b = (f(l, idx, dw, score, renormalise, 2.5) for f in (ref.route_backward, ref.route_backward_rows))
    assert np.allclose(a, b, rtol=1e-11, atol=1e-15)
