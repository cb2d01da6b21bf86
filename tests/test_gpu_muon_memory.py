"""Muon steps on other streams and in graphs, by objects that are gone before the step has run."""
import gc

import pytest
import torch

from gpu_util import mxq
from test_gpu_muon import inputs

pytestmark = pytest.mark.gpu

SHAPE = (4, 300, 500)  # a workspace of some megabytes


def tensors(seed=0):
    return [20 * inputs("noise", SHAPE, seed + 1)], [inputs("low_rank", SHAPE, seed + 2)], [inputs("noise", SHAPE, seed + 3)]


def after_steps(n):
    p, g, m = tensors()
    opt = mxq().Muon(p, g, m)
    for _ in range(n):
        opt.step(lr=0.02)
    torch.cuda.synchronize()
    return p[0], m[0]


def fill_what_is_free():
    """Memory that the current stream's pool hands out, overwritten."""
    size = mxq().mxq_orthogonalize_workspace(*SHAPE, 0)
    return [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]


@pytest.mark.parametrize("handle", ["stream", "integer", "current"])
def test_a_step_outlives_its_muon(handle):
    want = after_steps(1)
    p, g, m = tensors()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    if handle == "current":
        with torch.cuda.stream(st):
            mxq().Muon(p, g, m).step(lr=0.02)
    else:
        mxq().Muon(p, g, m).step(lr=0.02, stream=st if handle == "stream" else st.cuda_stream)
    gc.collect()
    filled = fill_what_is_free()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert torch.equal(p[0], want[0]) and torch.equal(m[0], want[1])
    assert all(bool((t == 0xFF).all()) for t in filled)


def test_a_graph_outlives_its_muon():
    p, g, m = tensors()
    start = [t[0].clone() for t in (p, m)]
    opt = mxq().Muon(p, g, m)
    opt.step(lr=0.02)  # (as a program warms up before it captures)
    p[0].copy_(start[0])
    m[0].copy_(start[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(lr=0.02)
    del opt
    gc.collect()
    for n in range(1, 4):
        filled = fill_what_is_free()
        graph.replay()
        torch.cuda.synchronize()
        want = after_steps(n)  # eager work between the replays
        assert torch.equal(p[0], want[0]) and torch.equal(m[0], want[1]), n
        assert all(bool((t == 0xFF).all()) for t in filled)


def test_steps_of_one_muon_on_two_streams():
    """One after the other, as its weights need, but with nothing between the workspaces."""
    want = after_steps(4)
    p, g, m = tensors()
    opt = mxq().Muon(p, g, m)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    last = torch.cuda.current_stream()
    for i in range(4):
        st = streams[i & 1]
        st.wait_stream(last)
        opt.step(lr=0.02, stream=st)
        last = st
    torch.cuda.current_stream().wait_stream(last)
    torch.cuda.synchronize()
    assert torch.equal(p[0], want[0]) and torch.equal(m[0], want[1])
