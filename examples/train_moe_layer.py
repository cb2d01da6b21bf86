"""Train one MoE layer with MXFP8 expert GEMMs on an MI355X.

    python examples/train_moe_layer.py [--steps 50] [--tokens 4096] [--hidden 512] [--ffn 256] [--experts 32] [--top-k 4]

A layer y = sum_k w_k x W[e_k] learns a random linear map.  A step runs, on one stream and without a host
synchronisation:

    forward   router logits (torch) -> route (experts, weights, expert order) -> dispatch -> row quantisation of X and
              dual-axis quantisation of W -> ragged-M GEMM -> combine
    backward  combine_backward -> row and token-axis quantisation -> ragged-M GEMM (dX) and ragged-K GEMM (dW) ->
              combine without weights (dX per token); route_backward -> router gradient (torch)
    update    AdamW: expert weights in fp32 with the bf16 copy that the quantiser reads and MXFP8 states, the router with
              fp32 states; the balance bias moves against each expert's load
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_grouped_gemm_mxq_amd import mxq  # noqa: E402


class MoELayer:
    def __init__(self, hidden, ffn, experts, top_k, n_group=4, topk_group=2, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.routing = dict(score="sigmoid", n_group=n_group, topk_group=topk_group, group_top=2, renormalise=True, scale=1.0)
        self.top_k, self.experts = top_k, experts
        self.router = torch.randn(hidden, experts, generator=g, device=device) * hidden ** -0.5
        self.bias = torch.zeros(experts, device=device)
        self.master = torch.randn(experts, hidden, ffn, generator=g, device=device) * hidden ** -0.5
        self.weight = self.master.to(torch.bfloat16)
        self.d_master, self.d_router = torch.zeros_like(self.master), torch.zeros_like(self.router)
        state = lambda p, fmt: ([mxq.adamw_state(p, fmt)], [mxq.adamw_state(p, fmt)])  # noqa: E731
        self.optimisers = [
            mxq.AdamW([self.master], [self.d_master], *state(self.master, mxq.MXQ_ADAMW_MXFP8), copies=[self.weight]),
            mxq.AdamW([self.router], [self.d_router], *state(self.router, mxq.MXQ_ADAMW_F32), decay_scales=[0.0]),
        ]

    def forward(self, x):
        """x bf16 [T][H] -> y bf16 [T][F]; keeps what the backward needs."""
        T, K = x.shape[0], self.top_k
        logits = x.float() @ self.router
        r = mxq.route(logits, K, bias=self.bias, **self.routing)
        rows = mxq.dispatch(x, r["slot"], T * K)
        qx, qw = mxq.quantize(rows, mxq.MXQ_AXIS_ROW), mxq.quantize_batched(self.weight)
        y_rows = mxq.grouped_gemm(mxq.MXQ_GG_RAGGED_M, qx["q_row"], qx["s_row"], qw["q_colT"], qw["s_colT"], r["group_end"])
        self.saved = (x, logits, r, rows, qw, y_rows)
        return mxq.combine(y_rows, r["slot"], r["weights"])

    def backward(self, dy):
        """dy bf16 [T][F] -> dx bf16 [T][H]; the weights' and the router's gradients into d_master and d_router."""
        x, logits, r, rows, qw, y_rows = self.saved
        d_rows, d_weights = mxq.combine_backward(dy, r["slot"], rows.shape[0], r["weights"], y_rows)
        qx = mxq.quantize_grouped(rows, r["group_end"])
        qd = mxq.quantize_grouped(d_rows, r["group_end"], mxq.MXQ_AXIS_ROW | mxq.MXQ_AXIS_COLT, ldq=qx["ldq"])
        dx_rows = mxq.grouped_gemm(mxq.MXQ_GG_RAGGED_M, qd["q_row"], qd["s_row"], qw["q_row"], qw["s_row"], r["group_end"])
        mxq.mxq_grouped_gemm(mxq.MXQ_GG_RAGGED_K, qx["q_colT"], qx["s_colT"], qd["q_colT"], qd["s_colT"], self.d_master,
                             r["group_end"])
        d_logits = mxq.route_backward(logits, r["idx"], d_weights, score="sigmoid", renormalise=True)
        torch.mm(x.float().t(), d_logits, out=self.d_router)
        dx = mxq.combine(dx_rows, r["slot"], dtype=torch.float32) + d_logits @ self.router.t()
        return dx.to(torch.bfloat16)

    def update(self, step, lr, balance=1e-3):
        for opt in self.optimisers:
            opt.step(lr=lr, step=step, seed=1, weight_decay=0.01)
        ends = self.saved[2]["group_end"]
        load = torch.diff(ends, prepend=ends.new_zeros(1)).float()
        self.bias += balance * torch.sign(load.mean() - load)
        return load


def train(steps=50, tokens=4096, hidden=512, ffn=256, experts=32, top_k=4, lr=2e-3, device="cuda", log=print):
    """Losses of the steps."""
    layer = MoELayer(hidden, ffn, experts, top_k, device=device)
    g = torch.Generator(device=device).manual_seed(1)
    target = torch.randn(hidden, ffn, generator=g, device=device) * hidden ** -0.5
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, hidden, generator=g, device=device).to(torch.bfloat16)
        y = layer.forward(x)
        error = y.float() - x.float() @ target
        layer.backward((error * (2.0 / ffn)).to(torch.bfloat16))  # per token; the optimiser does not mind the scale
        load = layer.update(step, lr)
        losses.append(error.square().mean())
        if log and (step == 1 or step % 10 == 0):
            log(f"step {step:4d}  loss {losses[-1].item():.4f}  largest load {load.max().item() / load.mean().item():.2f} of the mean")
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 50), ("tokens", 4096), ("hidden", 512), ("ffn", 256), ("experts", 32), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=2e-3)
    train(**vars(ap.parse_args()))
