"""The MoE layer of examples/train_moe_layer.py: it learns, its gradients are those of the layer in 64 bits within the
rounding of its operands, and a step of library calls recorded into a HIP graph replays to the eager results."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import mxq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_moe_layer", os.path.join(ROOT, "examples", "train_moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_layer_learns():
    losses = example().train(steps=60, tokens=2048, hidden=256, ffn=128, experts=16, top_k=4, log=None)
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]


def test_gradients_against_the_layer_in_64_bits():
    """Each GEMM operand is rounded to E4M3 (at most 2^-4 of a value), activations and row gradients to bf16 first
    (2^-8): a product is off by at most 2 * 2^-4 + 2 * 2^-8 + their product < 0.14 of its size, and so is a sum of
    products of its sum of sizes.  The router's gradient takes a product of that kind through sums of up to top_k terms
    that cancel, so it is compared by norm, against the sums of sizes as well."""
    mod = example()
    T, H, F, E, K = 300, 96, 64, 8, 2
    layer = mod.MoELayer(H, F, E, K, n_group=2, topk_group=1, seed=3)
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(T, H, generator=g).to(torch.bfloat16), torch.randn(T, F, generator=g).to(torch.bfloat16)
    y = layer.forward(x.cuda())
    dx = layer.backward(dy.cuda())
    idx = layer.saved[2]["idx"].cpu().long()

    xd = x.double().requires_grad_()
    wr, w = layer.router.double().cpu().requires_grad_(), layer.weight.double().cpu().requires_grad_()
    s = torch.sigmoid(xd @ wr).gather(1, idx)
    p = s / s.sum(1, keepdim=True)
    rows = torch.stack([torch.stack([xd[t] @ w[e] for e in idx[t]]) for t in range(T)])  # [T][K][F]
    out = (p[:, :, None] * rows).sum(1)
    out.backward(dy.double())

    def sizes():
        """The same sums of absolute values."""
        a, v, d = xd.detach().abs(), w.detach().abs(), dy.double().abs()
        pr = p.detach()
        yr = torch.stack([torch.stack([a[t] @ v[e] for e in idx[t]]) for t in range(T)])
        dw, dxs = torch.zeros_like(w), torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for k, e in enumerate(idx[t]):
                dw[e] += pr[t, k] * torch.outer(a[t], d[t])
                dxs[t] += pr[t, k] * (v[e] @ d[t])
        dp = (yr * d[:, None, :]).sum(2)  # [T][K]
        dl = torch.zeros(T, E, dtype=torch.float64)
        one = (1 - s.detach())
        dl.scatter_(1, idx, pr * (dp + (pr * dp).sum(1, keepdim=True)) * one)
        return (pr[:, :, None] * yr).sum(1), dw, dxs + dl @ wr.detach().abs().t(), a.t() @ dl

    sy, sw, sx, sr = sizes()
    for got, want, size in ((y, out.detach(), sy), (layer.d_master, w.grad, sw), (dx, xd.grad, sx), (layer.d_router, wr.grad, sr)):
        err = (got.double().cpu() - want).abs()
        assert bool((err <= 0.14 * size + 2.0 ** -8 * want.abs()).all())
        assert float(err.norm()) <= 0.14 * float(want.norm())  # and, rounding being random, by norm


def test_captured_step_replays_to_the_eager_results():
    """Route, dispatch, combine, both gradients and AdamW with its control in device memory: recorded once, replayed
    with new tokens, learning rate, step and seed, with eager work between."""
    m = mxq()
    T, H, E, K = 200, 256, 24, 3
    g = torch.Generator().manual_seed(5)
    logits = [torch.randn(T, E, generator=g).cuda() for _ in range(4)]
    tokens = [torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    param = torch.randn(T * K, H, generator=g).cuda()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    o = {"idx": i32(T, K), "weights": torch.zeros(T, K, device="cuda"), "group_end": i32(E), "row_token": i32(T * K), "slot": i32(T, K),
         "workspace": torch.zeros(m.mxq_expert_order_workspace(T, K, E), dtype=torch.uint8, device="cuda")}
    l, x = logits[0].clone(), tokens[0].clone()
    rows, y = torch.zeros(T * K, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    drows, dw, dl = torch.zeros(T * K, H, device="cuda"), torch.zeros(T, K, device="cuda"), torch.zeros(T, E, device="cuda")
    control = m.adamw_control(1e-3, 1)
    cfg = m.route_config(K, "softmax", 1, 1, 1, True, 1.0)

    def fresh():
        p = param.clone()
        s, t = m.adamw_state(p), m.adamw_state(p)
        return p, s, t, m.AdamW([p], [drows], [s], [t])

    def step(opt):
        m.mxq_route(l, cfg, o["idx"], o["weights"], None, o["group_end"], o["row_token"], o["slot"], o["workspace"])
        m.mxq_combine_backward(x, o["slot"], T * K, rows)
        m.mxq_combine(rows, o["slot"], o["weights"], y)
        m.mxq_combine_backward(y, o["slot"], T * K, drows, dw, o["weights"], rows)
        m.mxq_route_backward(l, cfg, o["idx"], dw, dl)
        opt.step(control=control)

    def run(state, go):
        seen = []
        for k in range(4):
            l.copy_(logits[k])
            x.copy_(tokens[k])
            m.adamw_control(1e-3 * (k + 1), k + 1, seed=k, out=control)
            torch.cuda.synchronize()
            go()
            torch.cuda.synchronize()
            seen.append([t.clone() for t in (o["idx"], o["weights"], o["group_end"], o["row_token"], o["slot"], rows, y, drows, dw, dl, state[0],
                                             *state[1], *state[2])])
            m.route(logits[3 - k], K)  # eager work between the replays
        return seen

    eager = fresh()
    want = run(eager, lambda: step(eager[3]))
    other = fresh()
    warm = fresh()
    step(warm[3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(other[3])
    got = run(other, graph.replay)
    for k, (a, b) in enumerate(zip(got, want)):
        assert all(torch.equal(s, t) for s, t in zip(a, b)), k
