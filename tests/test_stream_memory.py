"""Outputs and temporaries of a helper that is given a stream are allocated within that stream, and the call runs within
it: on the CPU, with a tensor type that passes for a device tensor and a library that does nothing."""
import contextlib

import pytest
import torch

from moe_grouped_gemm_mxq_amd import mxq

EVENTS = []  # in order: "within", "left", "made", "called"


class Dev(torch.Tensor):
    """Passes for a device tensor, and notes what is made like it."""
    is_cuda = True

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func.__name__ in ("new_empty", "empty_like"):
            EVENTS.append("made")
        return super().__torch_function__(func, types, args, kwargs or {})


class Library:
    """Entry points that do nothing and succeed."""

    def __getattr__(self, name):
        return lambda *a: 64 if name == "mxq_expert_order_workspace" else EVENTS.append("called") or 0


@contextlib.contextmanager
def on(stream, device):
    EVENTS.append("within")
    yield
    EVENTS.append("left")


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


T, E, K, H = 6, 16, 2, 32
SLOT = dev(T, K, dtype=torch.int32)
HELPERS = {
    "route": lambda st: mxq.route(dev(T, E), K, stream=st),
    "route without an order": lambda st: mxq.route(dev(T, E), K, order=False, stream=st),
    "expert_order": lambda st: mxq.expert_order(SLOT, E, stream=st),
    "route_backward": lambda st: mxq.route_backward(dev(T, E), SLOT, dev(T, K), stream=st),
    "combine": lambda st: mxq.combine(dev(T * K, H), SLOT, dev(T, K), stream=st),
    "combine_backward": lambda st: mxq.combine_backward(dev(T, H), SLOT, T * K, dev(T, K), dev(T * K, H), stream=st),
    "dispatch": lambda st: mxq.dispatch(dev(T, H), SLOT, T * K, stream=st),
}


G, R = 2, 64
END = dev(G, dtype=torch.int32)


def u8(*shape):
    return dev(*shape, dtype=torch.uint8)


def operand(rows, k=64):
    return u8(rows, k), u8(*mxq.scale_shape(rows, k // 32))


HELPERS |= {
    "quantize": lambda st: mxq.quantize(dev(R, R, dtype=torch.bfloat16), stream=st),
    "quantize_batched": lambda st: mxq.quantize_batched(dev(2, R, R, dtype=torch.bfloat16), stream=st),
    "quantize_grouped": lambda st: mxq.quantize_grouped(dev(R, R, dtype=torch.bfloat16), END, 3, 256, stream=st),
    "qdq_fp4": lambda st: mxq.qdq_fp4(dev(R, R), True, stream=st),
    "quantize_fp4": lambda st: mxq.quantize_fp4(dev(R, R), stream=st),
    "quantize_fp4_grouped": lambda st: mxq.quantize_fp4_grouped(dev(R, R), END, 256, stream=st),
    "qdq_fp4_ste": lambda st: mxq.qdq_fp4_ste(dev(R, R), want_codes=True, stream=st),
    "ste_backward_fp4": lambda st: mxq.ste_backward_fp4(dev(R, R), u8(R, R // 8), stream=st),
    "gemm": lambda st: mxq.gemm(*operand(R), *operand(R), stream=st),
    "grouped_gemm": lambda st: mxq.grouped_gemm(mxq.MXQ_GG_RAGGED_K, *operand(R, 256), *operand(R, 256), END, stream=st),
}


@pytest.fixture
def events(monkeypatch):
    empty = torch.empty

    def made(*a, **kw):
        EVENTS.append("made")
        return empty(*a, **kw).as_subclass(Dev)

    monkeypatch.setattr(mxq, "_on", on)
    monkeypatch.setattr(mxq, "_lib", Library())
    monkeypatch.setattr(mxq, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(torch, "empty", made)
    mxq.mxq_expert_order_workspace.cache_clear()
    EVENTS.clear()
    yield EVENTS
    mxq.mxq_expert_order_workspace.cache_clear()


@pytest.mark.parametrize("name", HELPERS)
def test_a_helpers_memory_is_its_streams(name, events):
    HELPERS[name](5)
    assert events[0] == "within" and events[-1] == "left" and events.count("within") == 1
    assert "made" in events and events.count("called") == 1
    events.clear()
    HELPERS[name](None)
    assert "within" not in events and "made" in events and events.count("called") == 1
