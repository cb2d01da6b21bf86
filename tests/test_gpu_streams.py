"""Helpers given a stream: their outputs are that stream's memory, and right."""
import pytest
import torch

from gpu_util import mxq

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


def tensors(x):
    return [t for v in (x.values() if isinstance(x, dict) else x if isinstance(x, tuple) else (x,)) for t in [v] if torch.is_tensor(t)]


def check(call, rows=None):
    """call(stream): with a Stream, with its handle, and on the current stream the same values; `rows`: of a first output
    that is written in part."""
    want = tensors(call(None))
    st = torch.cuda.Stream()
    for given in (st, st.cuda_stream):
        st.wait_stream(torch.cuda.current_stream())
        got = tensors(call(given))
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        assert all(stream_of(t) == st.cuda_stream for t in got)
        torch.cuda.current_stream().wait_stream(st)
        for i, (a, b) in enumerate(zip(got, want)):
            a, b = (a[rows], b[rows]) if i == 0 and rows is not None else (a, b)
            assert torch.equal(a, b)


def test_routing_and_combine():
    m = mxq()
    T, E, K, H = 300, 32, 4, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    logits, x = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    r = m.route(logits, K)
    y, dw = torch.randn(T * K, H, generator=g, device="cuda"), torch.randn(T, K, generator=g, device="cuda")
    check(lambda st: m.route(logits, K, stream=st))
    check(lambda st: m.route(logits, K, order=False, stream=st))
    check(lambda st: m.expert_order(r["idx"], E, stream=st))
    check(lambda st: m.route_backward(logits, r["idx"], dw, stream=st))
    check(lambda st: m.combine(y, r["slot"], r["weights"], stream=st))
    check(lambda st: m.combine_backward(x, r["slot"], T * K, r["weights"], y, stream=st))
    check(lambda st: m.dispatch(x, r["slot"], T * K, stream=st))


def test_quantisers_and_gemms():
    m = mxq()
    g = torch.Generator(device="cuda").manual_seed(2)
    x32 = torch.randn(256, 256, generator=g, device="cuda")
    x = x32.to(torch.bfloat16)
    ends = torch.tensor([100, 256], dtype=torch.int32, device="cuda")
    q, w, k = m.quantize(x), m.quantize_batched(x.view(2, 128, 256)), m.quantize_grouped(x, ends)
    y, mask = m.qdq_fp4_ste(x32)
    check(lambda st: m.quantize(x, stream=st))
    check(lambda st: m.quantize_batched(x.view(2, 128, 256), stream=st))
    check(lambda st: m.quantize_grouped(x, ends, m.MXQ_AXIS_ROW, stream=st))
    check(lambda st: m.qdq_fp4(x32, True, stream=st))
    check(lambda st: m.quantize_fp4(x32, stream=st))
    check(lambda st: m.qdq_fp4_ste(x32, want_codes=True, stream=st))
    check(lambda st: m.ste_backward_fp4(x32, mask, stream=st))
    check(lambda st: m.gemm(q["q_row"], q["s_row"], q["q_row"], q["s_row"], stream=st))
    check(lambda st: m.grouped_gemm(m.MXQ_GG_RAGGED_M, q["q_row"], q["s_row"], w["q_row"], w["s_row"], ends, stream=st))
    check(lambda st: m.grouped_gemm(m.MXQ_GG_RAGGED_K, k["q_colT"], k["s_colT"], k["q_colT"], k["s_colT"], ends, stream=st))
    # columns between the groups of a grouped operand need not be written: compared by what a product reads
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a, b = m.quantize_grouped(x, ends, stream=st), m.quantize_fp4_grouped(x32, ends, stream=st)
    assert all(stream_of(t) == st.cuda_stream for d in (a, b) for t in tensors(d))
    torch.cuda.current_stream().wait_stream(st)
    product = lambda d: m.grouped_gemm(m.MXQ_GG_RAGGED_K, d["q_colT"], d["s_colT"], d["q_colT"], d["s_colT"], ends)  # noqa: E731
    assert torch.equal(product(a), product(k))
