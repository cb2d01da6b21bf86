"""The calls that README.md shows, as they stand there."""
import os
import textwrap

import pytest
import torch

from gpu_util import mxq

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
T, E, K, H, N = 96, 16, 8, 256, 200  # tokens, experts, choices of a token, columns of the weights and rows


def block(after):
    """The indented lines after the one that begins with `after`."""
    lines = open(README).read().split("\n")
    at = next(i for i, s in enumerate(lines) if s.startswith(after)) + 2
    end = next(i for i in range(at, len(lines)) if not lines[i].startswith("    "))
    return textwrap.dedent("\n".join(lines[at:end]))


def normal(*shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale


def layer():
    return {"mxq": mxq(), "torch": torch, "logits": normal(T, E, seed=1), "bias": normal(E, seed=2, scale=0.01), "x": normal(T, H, seed=3).bfloat16()}


def test_forward():
    env = layer()
    env["w"] = mxq().quantize_batched(normal(E, H, N, seed=4, scale=H ** -0.5).bfloat16())
    exec(block("A forward of an MoE layer"), env)
    assert env["out"].shape == (T, N) and bool(env["out"].isfinite().all())


def test_the_same_in_blocks_of_128():
    """The step takes the gradient that the product before it wrote: of two operands that are off by 3.6% each (2-norm)."""
    env = layer()
    m = env["mxq"]
    w32 = normal(E, N, H, seed=4, scale=H ** -0.5)
    env |= {"w32": w32, "w": w32.bfloat16(), "dy": normal(T * K, N, seed=5).bfloat16(), "grad": torch.full_like(w32, float("nan")),
            "momentum": torch.zeros_like(w32)}
    exec(block("A forward of an MoE layer").split("q = ")[0], env)
    env["opt"] = m.Muon([w32], [env["grad"]], [env["momentum"]], copies=[env["w"]])
    was = w32.clone()
    exec(block("The same in blocks of 128"), env)
    ends = [0, *env["r"]["group_end"].tolist()]
    want = torch.stack([env["dy"][a:b].double().T @ env["rows"][a:b].double() for a, b in zip(ends, ends[1:])])
    assert float((env["grad"].double() - want).norm() / want.norm()) <= 0.051
    assert torch.equal(env["w"], w32.bfloat16()) and bool(w32.isfinite().all()) and not torch.equal(w32, was)
    assert env["y"].shape == (T * K, N)
