"""Router, expert order and the gradient of the weights against 64-bit references.

Weights: relative error at most (4 R + 40) half steps of fp32, R the spread of the row's logits: exp of a
difference x - max costs R from the difference and R from its scaling, in the numerator and in the sum, two
steps each for exp and for the quotient, and at most 22 additions follow one another in the sum (16 of a
lane's own, 6 across lanes)."""
import numpy as np
import pytest
import torch

import moe_reference as ref
from gpu_util import host, mxq

pytestmark = pytest.mark.gpu

U = ref.U32


def f64(t):
    return t.detach().cpu().double().numpy()


def logits_of(T, E, dtype, seed, masked=0.0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    x = (std * torch.randn(T, E, generator=g)).to(dtype)
    if masked and T:
        x[torch.rand(T, E, generator=g) < masked] = -float("inf")
        x[T // 2] = torch.finfo(dtype).min
    return x.cuda()


def spread(l):
    fine = np.where(np.isfinite(l) & (l > ref.LOWEST), l, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            r = np.nanmax(fine, 1) - np.nanmin(fine, 1)
    return np.nan_to_num(r)[:, None] + np.nan_to_num(np.nanmax(np.abs(np.nan_to_num(fine)), 1, initial=0))[:, None]


def check_route(x, K, bias=None, **kw):
    m = mxq()
    E = x.shape[1]
    got = m.route(x, K, bias=bias, **kw)
    idx, w = ref.route(f64(x), K, bias=None if bias is None else f64(bias), **kw)
    assert np.array_equal(host(got["idx"]), idx)
    gw = f64(got["weights"])
    assert np.array_equal(np.isnan(gw), np.isnan(w))
    fine = np.isfinite(w)
    tol = (4 * spread(f64(x)) + 40) * U * np.abs(w) + 2.0 ** -126
    assert np.all(np.abs(np.where(fine, gw - w, 0)) <= np.where(fine, tol, 0))
    ends, token, slot = ref.expert_order(idx, E)
    assert np.array_equal(host(got["group_end"]), ends)
    assert np.array_equal(host(got["row_token"]), token)
    assert np.array_equal(host(got["slot"]), slot)
    again = m.route(x, K, bias=bias, **kw)
    for k in got:
        if not (k == "weights" and np.isnan(gw).any()):
            assert torch.equal(got[k], again[k]), k


SIZES = [(0, 8, 2), (1, 1, 1), (1, 2, 2), (2, 31, 5), (3, 32, 32), (5, 33, 8), (63, 64, 1), (64, 65, 6), (65, 100, 3),
         (7, 160, 6), (129, 256, 8), (17, 500, 9), (9, 512, 8), (4, 1000, 32), (33, 1024, 16), (1000, 32, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route_sizes(T, E, K, score, dtype):
    x = logits_of(T, E, dtype, 7 * T + E)
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
    for b in (None, bias, torch.zeros_like(bias)):
        check_route(x, K, b, score=score, renormalise=True, scale=2.5)
    check_route(x, K, bias, score=score, renormalise=False, scale=1.0)


@pytest.mark.parametrize("E,n_group,topk_group,K", [(256, 8, 4, 8), (256, 8, 1, 8), (96, 3, 2, 7), (64, 64, 5, 5), (30, 2, 2, 4),
                                                   (1024, 16, 3, 12), (48, 6, 4, 20), (36, 4, 2, 3), (160, 8, 3, 6)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, n_group, topk_group, K, group_top, score):
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    for dtype, masked in ((torch.float32, 0.0), (torch.bfloat16, 0.0), (torch.float32, 0.3), (torch.bfloat16, 0.6)):
        x = logits_of(41, E, dtype, E + K, masked)
        bias = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
        for b in (None, bias, torch.zeros_like(bias)):
            check_route(x, K, b, renormalise=True, scale=1.0, **kw)


@pytest.mark.parametrize("T", [9, 4100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,K", [(64, 8, 3, 6), (256, 8, 4, 8), (96, 3, 2, 4), (512, 64, 20, 8)])
def test_route_groups_of_equal_totals(E, n_group, topk_group, K, score, T):
    """Rows of few distinct logits: groups tie for the last place, for the first, and all of them; some are masked."""
    g = torch.Generator().manual_seed(E)
    x = torch.randint(0, 2, (T, E), generator=g).float()
    x[0], x[1, E // 2:] = 0.25, 1.0
    x[2, : E // n_group * (n_group - topk_group + 1)] = -float("inf")
    x[3] = torch.arange(E) // (E // n_group) % 2
    zero = torch.zeros(E, device="cuda")
    few = T < 100  # the reference takes its time
    for dtype in (torch.float32, torch.bfloat16) if few else (torch.float32,):
        for b in (None, zero) if few else (zero,):
            for top in (1, 2) if few else (2,):
                check_route(x.to(dtype).cuda(), K, b, score=score, n_group=n_group, topk_group=topk_group, group_top=top,
                            renormalise=True, scale=1.0)


@pytest.mark.parametrize("T", [41, 4100])
@pytest.mark.parametrize("E,n_group,topk_group,K", [(128, 64, 1, 8), (64, 64, 2, 6), (32, 16, 1, 8), (32, 16, 2, 7), (64, 16, 1, 16)])
def test_route_groups_smaller_than_top_k(E, n_group, topk_group, K, T):
    """The kept groups' experts, each once, and -1 after them."""
    bias = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        x = logits_of(T, E, dtype, E + K)
        for b in (None, bias):
            check_route(x, K, b, score="sigmoid", n_group=n_group, topk_group=topk_group, group_top=1, renormalise=True, scale=1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_masks(score, renormalise):
    """Masked experts, rows with fewer experts than top_k, none at all, and the lowest values of both types."""
    for dtype in (torch.float32, torch.bfloat16):
        x = logits_of(64, 40, dtype, 3, 0.85)
        x[5] = -float("inf")
        x[6, 1:] = torch.finfo(torch.bfloat16).min
        bias = torch.linspace(-0.5, 0.5, 40).cuda()
        for b in (None, bias):
            check_route(x, 8, b, score=score, renormalise=renormalise)
            check_route(x, 8, b, score=score, renormalise=renormalise, n_group=5, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_not_finite(score):
    x = logits_of(8, 50, torch.float32, 4)
    x[1, 7] = float("nan")
    x[2, :] = float("nan")
    x[3, 9] = float("inf")
    x[4, 3] = float("nan")
    x[4, 20] = -float("inf")
    x[5, 10:12] = float("inf")
    bias = torch.linspace(0.3, -0.3, 50).cuda()
    for b in (None, bias):
        check_route(x, 6, b, score=score, renormalise=False)
        check_route(x, 6, b, score=score, renormalise=True, n_group=5, topk_group=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bias_not_finite(score):
    x = logits_of(70, 40, torch.float32, 6, 0.2)
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        bias = torch.linspace(0.2, -0.2, 40)
        bias[[3, 17]] = value
        check_route(x, 5, bias.cuda(), score=score)
        check_route(x, 5, bias.cuda(), score=score, n_group=4, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_that_underflow_keep_their_ratio(score):
    """A bias that forces experts whose scores are below fp32 (and, at -800, below fp64): softmax of the chosen logits."""
    for far in (-95.0, -800.0):
        x = torch.zeros(3, 32)
        x[:, 8:12] = far + torch.tensor([0.0, 1.0, -1.0, 0.5])
        x[2, 0] = float("inf") if score == "sigmoid" else 0.0  # a row that is taken to fp64
        bias = torch.zeros(32)
        bias[8:12] = 5.0
        got = mxq().route(x.cuda(), 4, score=score, bias=bias.cuda())
        for t in range(3):
            i = host(got["idx"])[t].astype(int)
            assert sorted(i) == [8, 9, 10, 11]
            want = np.exp(f64(x)[t, i] - far)
            want /= want.sum()
            assert np.all(np.abs(f64(got["weights"])[t] - want) <= (4 * 2 * abs(far) + 40) * U * want)


def test_route_ties_go_to_the_lowest_index():
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(5, 96, dtype=dtype, device="cuda")
        x[1, 40:] = 1.0
        x[2, ::3] = 2.0
        x[3] = torch.arange(96, device="cuda") // 7
        x[4, 95] = 1e-3
        for kw in ({}, {"n_group": 8, "topk_group": 3, "group_top": 2}, {"n_group": 4, "topk_group": 2}):
            for b in (None, torch.zeros(96, device="cuda"), torch.full((96,), 0.25, device="cuda")):
                for score in ("softmax", "sigmoid"):
                    check_route(x, 8, b, score=score, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_signed_zeros_are_equal(score):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.full((2, 64), -1.0, dtype=dtype, device="cuda")
        x[0, [3, 20, 41]] = torch.tensor([-0.0, 0.0, -0.0], dtype=dtype, device="cuda")
        x[1, ::5] = -0.0
        x[1, 60] = 0.0
        for b in (None, torch.zeros(64, device="cuda")):
            check_route(x, 3, b, score=score)
            check_route(x, 3, b, score=score, n_group=4, topk_group=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_close_keys(score):
    """Keys that differ by less than fp32 resolves: the bias undoes the scores' differences up to its own rounding."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(1, 64, generator=g)
    s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
    bias = (1.0 - s[0]).float()
    key = np.sort(f64(s[0]) + f64(bias))
    assert np.min(np.diff(key)) > 1e-13 and np.max(np.diff(key)) < 1e-7  # apart in 64 bits, not in 32
    check_route(x.cuda(), 8, bias.cuda(), score=score)
    check_route(x.cuda(), 8, bias.cuda(), score=score, n_group=8, topk_group=3, group_top=2)
    # among ordinary rows, and far-off scores
    rows = logits_of(33, 64, torch.float32, 5)
    rows[::4] = x.cuda()
    check_route(rows, 8, bias.cuda(), score=score, n_group=4, topk_group=2, group_top=2)
    check_route(rows * 40, 8, bias.cuda(), score=score)


def test_route_strides_and_alignment():
    base = logits_of(20, 200, torch.float32, 9)
    for lo, hi in ((0, 128), (1, 129), (3, 60), (8, 200)):
        for x in (base[:, lo:hi], base.to(torch.bfloat16)[:, lo:hi]):
            check_route(x, 4)
    check_route(base.to(torch.bfloat16)[::2, 5:37], 4)


def test_route_far_rows():
    """A row stride that takes the last row's offset past 32 bits."""
    x = torch.empty_strided((3, 64), (1 << 30, 1), dtype=torch.float32, device="cuda")
    x.copy_(logits_of(3, 64, torch.float32, 2))
    check_route(x, 8, score="sigmoid")
    d = torch.empty_strided((3, 64), (1 << 30, 1), dtype=torch.float32, device="cuda")
    m = mxq()
    idx = m.route(x, 8, order=False)["idx"]
    dw = torch.ones(3, 8, device="cuda")
    dw[:, 0] = 2.0
    m.mxq_route_backward(x, m.route_config(8), idx, dw, d)
    assert torch.equal(d, m.route_backward(x.contiguous(), idx, dw))


def test_route_on_another_stream():
    m = mxq()
    x = logits_of(500, 64, torch.float32, 8)
    want = m.route(x, 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = {k: torch.empty_like(v) for k, v in want.items()}
    got = m.route(x, 8, out=out, stream=st)
    st.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


# ------------------------------------------------------------------ expert order
@pytest.mark.parametrize("T,K,E", [(0, 1, 1), (1, 1, 1), (1, 8, 8), (127, 8, 3), (128, 8, 256), (129, 8, 256), (1024, 1, 1024),
                                  (2049, 5, 7), (5003, 8, 32), (40000, 2, 1000)])
def test_expert_order(T, K, E):
    m = mxq()
    g = torch.Generator().manual_seed(T + E)
    for kind in ("random", "one", "dropped"):
        if kind == "one":
            idx = torch.full((T, K), E - 1, dtype=torch.int32)
        elif kind == "random":
            idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
        else:  # out of range on both sides
            idx = torch.randint(-2, E + 3, (T, K), generator=g, dtype=torch.int32)
            if T:
                idx[0, 0] = -2 ** 31
                idx[-1, -1] = 2 ** 31 - 1
        got = m.expert_order(idx.cuda(), E)
        for name, want in zip(("group_end", "row_token", "slot"), ref.expert_order(idx.numpy(), E)):
            assert np.array_equal(host(got[name]), want), (kind, name)


def test_expert_order_of_many_chunks():
    m = mxq()
    idx = torch.randint(0, 77, (120000, 8), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    got = m.expert_order(idx.cuda(), 77)
    flat = idx.reshape(-1).numpy()
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(host(got["row_token"]), order // 8)
    slot = np.empty_like(order)
    slot[order] = np.arange(len(order))
    assert np.array_equal(host(got["slot"]).reshape(-1), slot)
    assert np.array_equal(host(got["group_end"]), np.cumsum(np.bincount(flat, minlength=77)))


# ------------------------------------------------------------------ gradient
def check_backward(x, idx, dw, score, renormalise, scale=1.0):
    """|err| <= (6 R + 64) half steps of s_e (sum_k |g_k| p_k + |g_e|): the factors of the weights' bound, with the
    sum over the chosen experts and two products more; bf16 results another half step of theirs."""
    m = mxq()
    got = f64(m.route_backward(x, idx, dw, score=score, renormalise=renormalise, scale=scale))
    l, i, g = f64(x), host(idx), f64(dw)
    want = ref.route_backward(l, i, g, score, renormalise, scale)
    E = l.shape[1]
    with np.errstate(all="ignore"):
        off = l <= ref.LOWEST
        s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - np.max(np.where(off, -np.inf, l), 1, keepdims=True))
    s = np.where(off, 0, s)
    if score == "softmax":
        s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    G = np.zeros_like(l)
    for t in range(len(l)):
        for k in range(i.shape[1]):
            if 0 <= i[t, k] < E and not off[t, i[t, k]]:
                G[t, i[t, k]] = abs(g[t, k]) * scale
    p = np.where(G > 0, s, 0)
    size = p * G if score == "sigmoid" and not renormalise else s * (G + (s * G).sum(1, keepdims=True))
    if renormalise:
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        size = p * (G + (p * G).sum(1, keepdims=True))
    tol = (6 * spread(l) + 64) * U * size + 2.0 ** -126
    if x.dtype == torch.bfloat16:
        tol = tol + ref.UBF16 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol)
    return got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route_backward(T, E, K, score, renormalise):
    m = mxq()
    for dtype, masked in ((torch.float32, 0.0), (torch.bfloat16, 0.0), (torch.float32, 0.4)):
        x = logits_of(T, E, dtype, T + E, masked)
        idx = m.route(x, K, score=score, order=False)["idx"]
        dw = torch.randn(T, K, generator=torch.Generator().manual_seed(E)).cuda()
        check_backward(x, idx, dw, score, renormalise, 2.5)


def test_route_backward_drops_bad_indexes():
    x = logits_of(6, 20, torch.float32, 1)
    idx = torch.tensor([[0, -1, 5], [20, 3, 1], [-2 ** 31, 2 ** 31 - 1, 19], [-1, -1, -1], [7, 8, 9], [1, 2, 40]], dtype=torch.int32).cuda()
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(2)).cuda()
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            check_backward(x, idx, dw, score, renormalise)


def test_route_backward_strides():
    m = mxq()
    base = logits_of(9, 100, torch.bfloat16, 3)
    x = base[:, 3:80]
    idx = m.route(x, 5, order=False)["idx"]
    dw = torch.randn(9, 5, generator=torch.Generator().manual_seed(2)).cuda()
    out = torch.full((9, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mxq_route_backward(x, m.route_config(5), idx, dw, out[:, 5:82])
    assert torch.equal(out[:, 5:82], m.route_backward(x.contiguous(), idx, dw))
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 82:] == 7).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward_against_differences(score, renormalise):
    """Central differences of the forward kernel.  Every weight's third derivative along one logit is below 6, so the
    difference is off by h^2 times sum |dw|, and by the weights' rounding over h."""
    m = mxq()
    E, K, h = 24, 4, 2.0 ** -7
    x = logits_of(1, E, torch.float32, 12)
    idx = m.route(x, K, score=score, order=False)["idx"]
    dw = torch.randn(1, K, generator=torch.Generator().manual_seed(3)).cuda()
    step = h * torch.eye(E, device="cuda")
    pinned = torch.zeros(E, device="cuda")
    pinned[idx[0].long()] = torch.arange(K, 0, -1, device="cuda") * 10.0  # the choice stays, whatever the logits
    w = [m.route(x + s * step, K, score=score, bias=pinned, renormalise=renormalise, order=False) for s in (1, -1)]
    assert all(bool((v["idx"] == idx).all()) for v in w)
    diff = ((w[0]["weights"].double() - w[1]["weights"].double()) * dw.double()).sum(1).cpu().numpy() / (2 * h)
    got = check_backward(x, idx, dw, score, renormalise)[0]
    total = float(dw.abs().sum())
    assert np.all(np.abs(diff - got) <= total * (h * h + (4 * 10 + 40) * U / h + 1e-5))


@pytest.mark.parametrize("T,E,K", [(5, 64, 4), (700, 96, 6)])
def test_route_into_the_callers_buffers(T, E, K):
    """The same buffers call after call, with a workspace that the first call puts there or the caller's own."""
    m = mxq()
    x = [logits_of(T, E, torch.float32, s) for s in (1, 2)]
    fresh = [m.route(v, K) for v in x]
    out = {k: torch.full_like(v, -9) for k, v in fresh[0].items()}
    own = dict(out, workspace=torch.full((m.mxq_expert_order_workspace(T, K, E),), 255, dtype=torch.uint8, device="cuda"))
    for buffers in (out, own):
        for v, want in zip(x, fresh):
            got = m.route(v, K, out=buffers)
            assert set(got) == set(want)
            for k in want:
                assert got[k] is buffers[k] and torch.equal(got[k], want[k]), k
        assert buffers["workspace"].numel() >= m.mxq_expert_order_workspace(T, K, E)


def group_totals(x, bias, score, n_group, group_top):
    """fp64 [T][n_group]: sums of each group's best keys (masked experts left out)."""
    off = x <= ref.LOWEST
    s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x - np.where(off, -np.inf, x).max(1, keepdims=True))
    s = np.where(off, 0, s)
    s = s if score == "sigmoid" else s / s.sum(1, keepdims=True)
    k = np.sort(np.where(off, -np.inf, s + bias).reshape(len(x), n_group, -1), axis=2)[:, :, -group_top:]
    return np.where(np.isinf(k), 0, k).sum(2)


@pytest.mark.parametrize("magnitude", [16.0, 128.0, 1e3, 1e4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,K,masked", [(64, 32, 7, 8, 0), (128, 64, 20, 6, 0), (16, 8, 3, 4, 0), (64, 8, 3, 4, 6),
                                                          (256, 16, 5, 8, 14)])
def test_route_groups_with_biases_of_both_signs(E, n_group, topk_group, K, masked, score, magnitude):
    """A group's best two keys are +magnitude and -magnitude: its total is small, but the keys are rounded at the
    magnitude.  Logits are drawn so close that the totals differ by about those roundings, and stay apart in 64 bits."""
    g = torch.Generator().manual_seed(E + int(magnitude))
    T, per = 200, E // n_group
    x = magnitude * 2.0 ** -20 * torch.randn(T, E, generator=g)
    bias = torch.where(torch.arange(per) % 2 == 0, magnitude, -magnitude).repeat(n_group)
    if masked:  # all but the last two of a group
        x.view(T, n_group, per)[:, :, :masked] = -float("inf")
    total = np.sort(group_totals(f64(x), f64(bias), score, n_group, 2), axis=1)[:, ::-1]
    gap = total[:, topk_group - 1] - total[:, topk_group]
    assert gap.min() > 16 * magnitude * 2.0 ** -53 and np.median(gap) < magnitude * 2.0 ** -22
    check_route(x.cuda(), K, bias.cuda(), score=score, n_group=n_group, topk_group=topk_group, group_top=2, renormalise=True, scale=1.0)


@pytest.mark.parametrize("T,E,n_group", [(6, 8, 2), (6, 64, 8), (6, 96, 3), (6, 256, 8), (4100, 64, 8)])
def test_route_groups_go_by_scores_where_logits_differ(T, E, n_group):
    """Without a bias, logits whose scores are one number in 64 bits: a sigmoid of 1, a softmax that underflows.  Groups of
    one total go by their index, the experts of the kept ones by their logits."""
    per = E // n_group
    g = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=g)
    x[1::2, 0], x[1::2, per] = 40.0, 45.0  # scores 1 and 1: the first group
    x[0, 0], x[0, per] = 30.0, 45.0        # apart in 64 bits
    x[2, 2], x[2, per] = 1e-3, 1e-3 + 2.0 ** -30
    for dtype in (torch.float32, torch.bfloat16) if T < 100 else (torch.float32,):
        for top in (1, 2):
            check_route(x.to(dtype).cuda(), 2, score="sigmoid", n_group=n_group, topk_group=1, group_top=top)
            check_route(x.to(dtype).cuda(), 5, score="sigmoid", n_group=n_group, topk_group=n_group - 1, group_top=top)
    x[1::2] *= 0.125
    x[1::2, :per] -= 900.0            # score 0
    x[1::2, per:2 * per] -= 800.0     # score 0
    x[3, :per] += 300.0               # not 0 in 64 bits, 0 in 32
    x[5, 1] = float("nan")
    for topk_group in (1, n_group - 1):
        for top in (1, 2):
            check_route(x.cuda(), 2, score="softmax", n_group=n_group, topk_group=topk_group, group_top=top, renormalise=True)
    for far in (5.0, 40.0, 400.0):  # scores from ordinary ones to those of 0 and 1
        for score in ("softmax", "sigmoid"):
            check_route((far * torch.randn(T, E, generator=g)).cuda(), 4, score=score, n_group=n_group, topk_group=n_group - 1, renormalise=True)
    close = 1.0 + 2.0 ** -23 * torch.randint(0, 3, (T, E), generator=g) * torch.tensor([1.0, 2.0 ** -10, 2.0 ** -20, 0.0]).repeat(E // 4)
    for score in ("softmax", "sigmoid"):
        check_route(close.cuda(), 4, score=score, n_group=n_group, topk_group=n_group - 1)
        check_route((close - 1.0).cuda(), 4, score=score, n_group=n_group, topk_group=n_group - 1)
    if n_group > 2:  # exp(-744.9) is the least number of 64 bits, and 0 after the division by the sum
        x = torch.full((T, E), -900.0)
        x[:, 0], x[:, per], x[:, 2 * per:3 * per] = -746.5, -744.9, 0.0
        for top in (1, 2):
            check_route(x.cuda(), 3, score="softmax", n_group=n_group, topk_group=2, group_top=top)
            check_route(x.cuda(), min(per + 2, 32), score="softmax", n_group=n_group, topk_group=2, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_of_keys_that_overflow_when_added(score):
    """Best two keys of 3e38 of one sign: their total is past fp32, and finite in 64 bits."""
    x = logits_of(50, 16, torch.float32, 21)
    bias = torch.tensor([-3e38, -3e38, 0, 0, 3e38, 3e38, -3.4e38, -3e38, 3e38, 2.5e38, -3e38, 1, 0, 0, -3e38, -3e38])
    for topk_group in range(1, 9):
        for top in (1, 2):
            for b in (bias, -bias):
                check_route(x, 16, b.cuda(), score=score, n_group=8, topk_group=topk_group, group_top=top)


# ------------------------------------------------------------------ many rows: other shapes of the kernels
def row_spread(l):
    """spread of rows, vectorised: range of the unmasked logits and their largest magnitude."""
    off = l <= ref.LOWEST
    some = ~off.all(1)
    hi, lo = (np.where(some, f(np.where(off, o, l), axis=1), 0.0) for f, o in ((np.max, -np.inf), (np.min, np.inf)))
    return (hi - lo + np.maximum(np.abs(hi), np.abs(lo)))[:, None]


def check_route_rows(x, K, bias=None, **kw):
    E = x.shape[1]
    got = mxq().route(x, K, bias=bias, **kw)
    idx, w = ref.route_rows(f64(x), K, bias=None if bias is None else f64(bias), **kw)
    assert np.array_equal(host(got["idx"]), idx)
    assert np.all(np.abs(f64(got["weights"]) - w) <= (4 * row_spread(f64(x)) + 40) * U * np.abs(w) + 2.0 ** -126)
    for name, want in zip(("group_end", "row_token", "slot"), ref.expert_order(idx, E)):
        assert np.array_equal(host(got[name]), want), name


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,n_group", [(4099, 40, 20, 1), (4099, 100, 6, 1), (4099, 256, 8, 1), (4099, 256, 8, 8), (4099, 200, 20, 1),
                                           (4099, 300, 8, 1), (4099, 512, 8, 1), (4099, 512, 8, 8), (4099, 1000, 8, 1), (2000, 1024, 8, 1),
                                           (65536, 32, 8, 1), (33000, 256, 2, 1), (5003, 32, 8, 4)])
def test_route_many_rows(T, E, K, n_group, score):
    """Rows held by 16, 32 and 64 lanes with up to 16 experts each, and the expert order by either way."""
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
    for dtype, b, masked in ((torch.float32, bias, 0.0), (torch.float32, None, 0.1), (torch.bfloat16, bias, 0.1), (torch.bfloat16, None, 0.0)):
        kw = dict(n_group=n_group, topk_group=max(1, n_group // 2), group_top=2) if n_group > 1 else {}
        check_route_rows(logits_of(T, E, dtype, T + E + K, masked), K, b, score=score, renormalise=b is not None, scale=2.5, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("T,E,K", [(4099, 40, 5), (4099, 100, 6), (4099, 256, 8), (4099, 255, 16), (4099, 256, 20), (4099, 300, 8),
                                   (4099, 512, 8), (16390, 256, 8)])
def test_route_backward_many_rows(T, E, K, score, renormalise):
    """The bounds of check_backward, on all rows at once."""
    for dtype, masked in ((torch.float32, 0.0), (torch.bfloat16, 0.2)):
        x = logits_of(T, E, dtype, T + E, masked)
        idx = mxq().route(x, K, score=score, order=False)["idx"]
        dw = torch.randn(T, K, generator=torch.Generator().manual_seed(E)).cuda()
        got = f64(mxq().route_backward(x, idx, dw, score=score, renormalise=renormalise, scale=2.5))
        l, i, g = f64(x), host(idx), f64(dw)
        want = ref.route_backward_rows(l, i, g, score, renormalise, 2.5)
        off, there = l <= ref.LOWEST, i >= 0
        with np.errstate(all="ignore"):
            s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - np.where(off, -np.inf, l).max(1, keepdims=True))
        s = np.where(off, 0, s)
        if score == "softmax":
            s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
        G, named = np.zeros((T, E + 1)), np.zeros((T, E + 1), bool)
        np.put_along_axis(G, np.where(there, i, E), np.abs(g) * 2.5, 1)
        np.put_along_axis(named, np.where(there, i, E), True, 1)
        G, named = G[:, :E], named[:, :E]
        if renormalise:
            p = np.where(named, s, 0)
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
            size = p * (G + (p * G).sum(1, keepdims=True))
        elif score == "sigmoid":
            size = s * G
        else:
            size = s * (G + (s * G).sum(1, keepdims=True))
        tol = (6 * row_spread(l) + 64) * U * size + 2.0 ** -126 + (ref.UBF16 * np.abs(want) if dtype == torch.bfloat16 else 0)
        assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("seed", range(16))
def test_route_random(seed):
    """Twelve routings of random sizes, groups, types, masks and biases from none to a thousand."""
    rng = np.random.default_rng(seed)
    for _ in range(12):
        n_group = int(rng.choice([1, 1, 2, 3, 4, 8, 16, 64]))
        per = int(np.exp(rng.uniform(0, np.log(1024 / n_group))))
        E = n_group * per
        T, K = int(np.exp(rng.uniform(0, np.log(6000)))), int(rng.integers(1, min(E, 32) + 1))
        dtype = (torch.float32, torch.bfloat16)[rng.integers(2)]
        size = float(rng.choice([0.0, 0.0, 0.1, 1.0, 30.0, 1000.0]))
        bias = torch.from_numpy(size * rng.standard_normal(E)).float().cuda() if size else None
        kw = dict(score=("softmax", "sigmoid")[rng.integers(2)], n_group=n_group, topk_group=int(rng.integers(1, n_group + 1)),
                  group_top=int(rng.integers(1, 3)), renormalise=bool(rng.integers(2)))
        x = logits_of(T, E, dtype, int(rng.integers(1 << 30)), float(rng.choice([0.0, 0.0, 0.3, 0.8])), float(rng.choice([0.3, 1.5, 5.0])))
        print(T, E, K, dtype, size, kw, flush=True)
        check_route_rows(x, K, bias, **kw)
