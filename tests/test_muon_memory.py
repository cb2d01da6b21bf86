"""Whose memory a Muon step works in: the stream's that it runs on, given back when the step has been queued."""
import contextlib

import pytest
import torch

from moe_grouped_gemm_mxq_amd import mxq
from test_block128_muon_refusals import Dev, dev, library  # noqa: F401  (library: a fixture)


@pytest.fixture
def events(library, monkeypatch):  # noqa: F811
    """What a step does, in order: enters and leaves a stream, allocates, calls."""
    seen = []

    @contextlib.contextmanager
    def on(stream, device):
        seen.append(("within", stream))
        yield
        seen.append("left")

    empty = torch.empty

    def made(*a, **kw):
        seen.append("made")
        return empty(*a, **kw).as_subclass(Dev)

    muon = mxq.mxq_muon

    def called(param, grad, m, cfg, workspace, copy=None, control=None, stream=None):
        seen.append("step")
        muon(param, grad, m, cfg, workspace, copy, control, stream)

    monkeypatch.setattr(mxq, "_on", on)
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(mxq, "mxq_muon", called)
    return seen


def tensors(*shapes):
    return [[dev(*s) for s in shapes] for _ in range(3)]


def test_the_workspace_is_the_given_streams(events, library):  # noqa: F811
    opt = mxq.Muon(*tensors((4, 5), (2, 6, 7)))
    events.clear()
    opt.step(stream=5)
    assert events == [("within", 5), "made", "step", "step", "left"] and library == ["mxq_muon"] * 2


def test_the_workspace_is_the_current_streams(events):
    opt = mxq.Muon(*tensors((4, 5)))
    events.clear()
    opt.step()
    opt.step()  # (perhaps on another stream)
    assert events == ["made", "step"] * 2


def test_a_muon_holds_no_workspace(events):
    opt = mxq.Muon(*tensors((4, 5)))
    assert events == [] and not any(isinstance(v, torch.Tensor) for v in vars(opt).values())


def test_no_tensors(events):
    mxq.Muon([], [], []).step(stream=5)
    assert events == []
