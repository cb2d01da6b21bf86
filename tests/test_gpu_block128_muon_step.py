"""The block-128 operators and Muon as they are used together: an MoE layer's training step, eager, on streams and in graphs."""
import numpy as np
import pytest
import torch

import muon_reference as muon
from gpu_util import mxq
from test_gpu_muon import SINGLE, TRIPLE, inputs, off, rounding, wide
from test_gpu_streams import check

pytestmark = pytest.mark.gpu


def normal(*shape, seed, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


class Layer:
    """out = sum_k w_k W2[e_k] (W1[e_k] x) of the tokens' top experts, with FP8 products both ways, and a Muon step."""
    E, K, T, H, F = 8, 2, 300, 256, 200

    def __init__(self, seed=0):
        m = mxq()
        E, T, H, F = self.E, self.T, self.H, self.F
        self.w = [normal(E, F, H, seed=seed + 1, dtype=torch.float32, scale=H ** -0.5), normal(E, H, F, seed=seed + 2, dtype=torch.float32, scale=F ** -0.5)]
        self.copies = [w.bfloat16() for w in self.w]
        self.grads, self.m = [torch.zeros_like(w) for w in self.w], [torch.zeros_like(w) for w in self.w]
        self.x, self.logits, self.target = normal(T, H, seed=seed + 3), normal(T, E, seed=seed + 4, dtype=torch.float32), normal(T, H, seed=seed + 5)
        self.out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.dx = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.opt = m.Muon(self.w, self.grads, self.m, self.copies)

    def step(self):
        m, rows = mxq(), self.T * self.K
        r = m.route(self.logits, self.K)
        slot, ends, weights = r["slot"], r["group_end"], r["weights"]
        q = [m.quantize128(c, 3, 128) for c in self.copies]
        x = m.dispatch(self.x, slot, rows)
        qx = m.quantize128(x)
        h = m.grouped_gemm128(0, qx["q_row"], qx["s_row"], q[0]["q_row"], q[0]["s_row"], ends)
        qh = m.quantize128(h)
        y = m.grouped_gemm128(0, qh["q_row"], qh["s_row"], q[1]["q_row"], q[1]["s_row"], ends)
        self.out.copy_(m.combine(y, slot, weights, dtype=torch.bfloat16))
        dout = self.out - self.target
        dy, _ = m.combine_backward(dout, slot, rows, weights, y)
        # gradients of rows: rows of dY against the weights' transposes; of weights: both operands' token axes
        gdy = m.quantize128_grouped(dy, ends, 3)
        gh = m.quantize128_grouped(h, ends)
        self.grads[1].copy_(m.grouped_gemm128(1, gdy["q_colT"], gdy["s_colT"], gh["q_colT"], gh["s_colT"], ends, dtype=torch.float32))
        dh = m.grouped_gemm128(0, gdy["q_row"], gdy["s_row"], q[1]["q_colT"], q[1]["s_colT"], ends)
        gdh, gx = m.quantize128_grouped(dh, ends, 3), m.quantize128_grouped(x, ends)
        m.mxq_grouped_gemm128(1, gdh["q_colT"], gdh["s_colT"], gx["q_colT"], gx["s_colT"], self.grads[0], ends)
        dx = m.grouped_gemm128(0, gdh["q_row"], gdh["s_row"], q[0]["q_colT"], q[0]["s_colT"], ends)
        self.dx.copy_(m.combine(dx, slot, dtype=torch.bfloat16))
        self.opt.step(lr=0.02, weight_decay=0.01)
        return r

    def state(self):
        return [*self.w, *self.copies, *self.grads, *self.m, self.out, self.dx]


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_training_step_against_the_formulas():
    """The layer's results and gradients against 64 bits.  An operand is off by at most 2^-4 of itself where its code is
    normal, uniformly within a code's step: 2^-4 / sqrt(3) = 3.6% root mean square at the worst value, and the errors of
    the 200 or more terms of a sum are independent, so a product of two such operands is off by at most
    sqrt(2) 3.6% = 5.1% of its 2-norm, and one whose operand is such a product and is quantised again, by at most
    sqrt(5.1^2 + 2 3.6^2) = 7.2%; a third product in a row, 8.9%."""
    layer = Layer()
    w1, w2 = (w.double() for w in layer.w)
    r = layer.step()
    x, logits, target = layer.x.double(), layer.logits.double(), layer.target.double()
    idx, weights = r["idx"].long(), r["weights"].double()
    h = torch.stack([x @ w1[e].T.contiguous() for e in range(layer.E)])  # [E][T][F]
    t = torch.arange(layer.T, device="cuda")[:, None].expand_as(idx)
    hk = h[idx, t]  # [T][K][F]
    y = torch.stack([torch.stack([w2[int(e)] @ v for e, v in zip(es, vs)]) for es, vs in zip(idx, hk)])
    out = (weights[..., None] * y).sum(1)
    assert relative(layer.out, out) <= 0.072 + 2 ** -8
    dy = weights[..., None] * (layer.out.double() - target)[:, None]  # (of the output as it was rounded: dout is an input to what follows)
    g2, g1, dx = torch.zeros_like(w2), torch.zeros_like(w1), torch.zeros_like(x)
    for e in range(layer.E):
        at = (idx == e).nonzero()
        a, d, xs = hk[at[:, 0], at[:, 1]], dy[at[:, 0], at[:, 1]], x[at[:, 0]]
        g2[e] = d.T @ a
        dh = d @ w2[e]
        g1[e] = dh.T @ xs
        dx.index_add_(0, at[:, 0], dh @ w1[e])
    assert relative(layer.grads[1], g2) <= 0.072
    assert relative(layer.grads[0], g1) <= 0.072
    assert relative(layer.dx, dx) <= 0.072 + 2 ** -8
    # the step of the weights, from the gradients that it was given
    for w, copy, g, mom, was in zip(layer.w, layer.copies, layer.grads, layer.m, (w1, w2)):
        scale = mxq().muon_scale(w.shape)
        for e in range(layer.E):
            want, want_m, o = muon.step(wide(was[e]), wide(g[e]), np.zeros(was[e].shape), lr=0.02, momentum=0.95, nesterov=True, weight_decay=0.01, scale=scale)
            assert off(wide(mom[e]), want_m) <= 4 * 2.0 ** -24
            tol = TRIPLE * 0.02 * scale * np.linalg.norm(o) + 2.0 ** -22 * np.linalg.norm(want)
            assert np.linalg.norm(wide(w[e]) - want) <= tol
        assert torch.equal(copy, w.bfloat16())


def test_captured_steps_replay_to_the_eager_ones():
    eager, captured, other = Layer(), Layer(), Layer(50)
    captured.step()
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    torch.cuda.synchronize()
    for rep in range(3):
        graph.replay()
        other.step()  # eager work of another layer between the replays
        eager.step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured.state(), eager.state())):
            assert torch.equal(a, b), (rep, i)
    captured.step()  # and eagerly again
    eager.step()
    assert all(torch.equal(a, b) for a, b in zip(captured.state(), eager.state()))


def test_two_steps_at_once():
    """Two layers on two streams, over and over, as each alone."""
    alone, both = [Layer(), Layer(50)], [Layer(), Layer(50)]
    for layer in alone:
        for _ in range(4):
            layer.step()
    streams = [torch.cuda.Stream() for _ in both]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for st, layer in zip(streams, both):
            with torch.cuda.stream(st):
                layer.step()
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))


def test_given_streams():
    m = mxq()
    x, w, ends = normal(300, 256, seed=1), normal(2, 130, 256, seed=2), torch.tensor([100, 300], dtype=torch.int32, device="cuda")
    q, k, one, e = m.quantize128(x, 3), m.quantize128_grouped(x, ends), m.quantize128(w[0], 1, 128), m.quantize128(w, 1, 128)
    check(lambda st: m.quantize128(x, 3, stream=st))
    check(lambda st: m.quantize128(w, 3, 128, stream=st))
    check(lambda st: m.quantize128_grouped(x, ends, m.MXQ_AXIS_ROW, stream=st))
    check(lambda st: m.gemm128(q["q_row"], q["s_row"], one["q_row"], one["s_row"], stream=st))
    check(lambda st: m.grouped_gemm128(0, q["q_row"], q["s_row"], e["q_row"], e["s_row"], ends, stream=st))
    check(lambda st: m.grouped_gemm128(1, k["q_colT"], k["s_colT"], k["q_colT"], k["s_colT"], ends, stream=st))
    check(lambda st: m.orthogonalize(w, stream=st))
    # steps on a stream that is given
    a, b = Layer(), Layer()
    a.opt.step(lr=0.1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b.opt.step(lr=0.1, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(p, q) for p, q in zip(a.state(), b.state()))


# (batch, R, C): 128 x 128 tiles, 256 x 256 ones with a last round in quarters (530 = 2 * 256 + 18 tiles), and large matrices
BIG = [((300, 100, 120), "noise"), ((530, 200, 300), "decay"), ((530, 300, 200), "noise"), ((2100, 2200), "noise"), ((4500, 1100), "noise")]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,kind", BIG)
def test_large_orthogonalisations(shape, kind, out):
    """fp32 sums over K of up to K / 16 terms of sixteen: as many roundings of 2^-23 in each of five iterations."""
    x = normal(*shape, seed=1, dtype=torch.float32) if kind == "noise" else inputs(kind, (2, *shape[1:]), 1).repeat(shape[0] // 2, 1, 1)
    got = mxq().orthogonalize(x, dtype=out).view(-1, *shape[-2:])
    x = x.view(-1, *shape[-2:])
    tol = (SINGLE if out == torch.bfloat16 else TRIPLE) + rounding(out) + 5 * max(shape[-2:]) / 16 * 2.0 ** -23
    for i in sorted({0, 1, len(x) // 2, len(x) - 3, len(x) - 1} & set(range(len(x)))):
        e = off(wide(got[i]), muon.orthogonalize(wide(x[i])))
        assert e <= tol, (i, e)


def test_norms_past_fp32s_range_of_reciprocals():
    x = inputs("noise", (40, 90), 1) * 1e-33  # a norm of 6e-35, whose reciprocal times the scale of X is past fp32's range
    for eps in (0.0, 1e-40):
        assert off(wide(mxq().orthogonalize(x, eps=eps, dtype=torch.float32)), muon.orthogonalize(wide(x), eps=eps)) <= TRIPLE


def test_in_place_and_extreme_updates():
    m = mxq()
    x = inputs("noise", (2, 100, 70), 4)
    want = m.orthogonalize(x, dtype=torch.float32)
    ws = torch.empty(m.mxq_orthogonalize_workspace(2, 100, 70, 0), dtype=torch.uint8, device="cuda")
    m.mxq_orthogonalize(x, m.newton_schulz(), x, ws)  # the matrix is read before the result is written
    assert torch.equal(x, want)
    # a rate of zero leaves the weights, and the momentum goes on
    p, g, mom = normal(100, 70, seed=1, dtype=torch.float32), inputs("noise", (100, 70), 2), torch.zeros(100, 70, device="cuda")
    was = p.clone()
    m.Muon([p], [g], [mom]).step(lr=0.0)
    assert torch.equal(p, was) and off(wide(mom), 0.05 * wide(g)) <= 4 * 2.0 ** -24
    # a gradient of zero without momentum only decays the weights
    m.Muon([p], [torch.zeros_like(g)], [torch.zeros_like(mom)]).step(lr=0.1, weight_decay=0.5)
    assert off(wide(p), 0.95 * wide(was)) <= 2.0 ** -23
