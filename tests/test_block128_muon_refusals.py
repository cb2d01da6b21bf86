"""Arguments that the block-128 quantisers and products and the Muon entry points refuse, on the host: no GPU is reached."""
import contextlib
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from moe_grouped_gemm_mxq_amd import mxq

INVALID, DEVICE = 1, 3
FAKE = 0x10000  # never dereferenced: the checks end first
HAS_GPU = torch.cuda.device_count() > 0
NAN, INF = float("nan"), float("inf")


def refused(status, says):
    assert status == INVALID
    assert says in mxq.mxq_last_error()


def call(name, defaults, kw):
    assert set(kw) <= set(defaults)
    return getattr(mxq._lib, name)(*(defaults | kw).values())


QUANTIZE = dict(x=FAKE, dt=1, batch=1, R=200, C=300, ldx=300, x_stride=0, tile=1, axis_mask=3, q_row=FAKE, s_row=FAKE, q_colT=FAKE,
                s_colT=FAKE, st=None)


@pytest.mark.parametrize("kw,says", [
    (dict(x=None), "NULL"), (dict(dt=2), "type"), (dict(dt=-1), "type"), (dict(batch=-1), "batch"), (dict(batch=65536), "batch"),
    (dict(R=-1), "rows"), (dict(R=2 ** 31), "rows"), (dict(C=0), "columns"), (dict(C=2 ** 31 - 128), "columns"), (dict(ldx=299), "ldx"),
    (dict(batch=2, x_stride=59999), "x_stride"), (dict(batch=2, x_stride=-1), "x_stride"), (dict(tile=0), "tile"), (dict(tile=64), "tile"),
    (dict(axis_mask=0), "axis_mask"), (dict(axis_mask=4), "axis_mask"), (dict(axis_mask=-1), "axis_mask"),
    (dict(q_row=None), "row outputs"), (dict(s_row=None), "row outputs"), (dict(q_colT=None), "colT outputs"), (dict(s_colT=None), "colT outputs"),
    (dict(x=FAKE + 1), "aligned"), (dict(x=FAKE + 2, dt=0), "aligned"), (dict(q_row=FAKE + 8), "16-byte"), (dict(q_colT=FAKE + 4), "16-byte"),
    (dict(s_row=FAKE + 2), "4-byte"), (dict(s_colT=FAKE + 1), "4-byte"),
])
def test_quantize128(kw, says):
    refused(call("mxq_quantize128", QUANTIZE, kw), says)


GROUPED = dict(x=FAKE, dt=1, T=200, C=300, ldx=300, group_end=FAKE, G=3, ldq=640, axis_mask=3, q_row=FAKE, s_row=FAKE, q_colT=FAKE, s_colT=FAKE,
               st=None)


@pytest.mark.parametrize("kw,says", [
    (dict(x=None), "NULL"), (dict(dt=7), "type"), (dict(T=-1), "rows"), (dict(T=2 ** 31), "rows"), (dict(C=0), "columns"), (dict(ldx=0), "ldx"),
    (dict(group_end=None), "group_end"), (dict(group_end=FAKE + 2), "group_end"), (dict(G=0), "G must"), (dict(G=1025), "G must"),
    (dict(ldq=0), "ldq"), (dict(ldq=-128), "ldq"), (dict(ldq=192), "ldq"), (dict(axis_mask=0), "axis_mask"), (dict(q_colT=None), "colT"),
    (dict(s_row=None), "row outputs"), (dict(q_colT=FAKE + 8), "16-byte"),
])
def test_quantize128_grouped(kw, says):
    refused(call("mxq_quantize128_grouped", GROUPED, kw), says)


def test_columns_of_grouped_operands():
    for T, G in ((0, 1), (1, 1), (1000, 8), (131072, 32), (2 ** 31 - 1, 1024)):
        n = mxq.mxq_grouped128_cols_max(T, G)
        assert n % 256 == 128 and T + 127 * G <= n < T + 127 * G + 384
    for T, G in ((-1, 4), (4, -1), (2 ** 31, 4)):
        assert mxq.mxq_grouped128_cols_max(T, G) == 0


GEMM = dict(A=FAKE, sA=FAKE, B=FAKE, sB=FAKE, b_tile=128, C=FAKE, cdt=1, M=5, N=300, K=256, ldc=300, st=None)
OPERANDS = [
    (dict(A=None), "NULL"), (dict(sA=None), "NULL"), (dict(B=None), "NULL"), (dict(sB=None), "NULL"), (dict(C=None), "NULL"), (dict(cdt=2), "type"),
    (dict(M=-1), "M must"), (dict(M=2 ** 31), "M must"), (dict(N=0), "N in"), (dict(N=2 ** 31), "N in"), (dict(K=0), "multiple of 128"),
    (dict(K=-128), "multiple of 128"), (dict(K=192), "multiple of 128"), (dict(K=1 << 23), "MXQ_GEMM_MAX_ROW_BYTES"), (dict(A=FAKE + 8), "16-byte"),
    (dict(B=FAKE + 1), "16-byte"), (dict(sA=FAKE + 2), "4-byte"), (dict(sB=FAKE + 1), "4-byte"), (dict(C=FAKE + 1), "elements"),
    (dict(C=FAKE + 2, cdt=0), "elements"),
]


@pytest.mark.parametrize("kw,says", OPERANDS + [(dict(ldc=299), "ldc"), (dict(b_tile=0), "b_tile"), (dict(b_tile=32), "b_tile")])
def test_gemm128(kw, says):
    refused(call("mxq_gemm128", GEMM, kw), says)


GROUPED_GEMM = dict(mode=0, A=FAKE, sA=FAKE, B=FAKE, sB=FAKE, C=FAKE, cdt=1, M=5, N=300, K=256, group_end=FAKE, G=2, st=None)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("kw,says", OPERANDS + [(dict(mode=2), "mode"), (dict(mode=-1), "mode"), (dict(G=0), "G must"), (dict(G=1025), "G must"),
                                                (dict(group_end=None), "group_end"), (dict(group_end=FAKE + 2), "group_end")])
def test_grouped_gemm128(kw, says, mode):
    refused(call("mxq_grouped_gemm128", GROUPED_GEMM, dict(mode=mode) | kw), says)


def iteration(**kw):
    c = mxq.newton_schulz()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


ROOM = mxq.mxq_orthogonalize_workspace(2, 40, 50, 1)
ORTHOGONALIZE = dict(x=FAKE, dt=0, batch=2, R=40, C=50, cfg=None, out=FAKE, odt=1, workspace=FAKE, nbytes=ROOM, st=None)
CONFIGS = [
    (dict(steps=0), "steps"), (dict(steps=33), "steps"), (dict(steps=-1), "steps"), (dict(a=NAN), "finite"), (dict(b=INF), "finite"),
    (dict(c=-INF), "finite"), (dict(a=65.0), "coefficients"), (dict(c=-65.0), "coefficients"), (dict(a=2.0, b=0.0, c=0.0), "coefficients"),
    (dict(a=3.4445, b=-4.775, c=3.0), "coefficients"), (dict(a=0.0, b=0.0, c=0.5), "coefficients"), (dict(eps=-1e-9), "eps"),
    (dict(eps=NAN), "eps"), (dict(eps=INF), "eps"),
]
MATRICES = [
    (dict(batch=-1), "batch"), (dict(batch=65536), "batch"), (dict(R=0), "R and C"), (dict(C=0), "R and C"), (dict(R=2 ** 20 + 1), "R and C"),
    (dict(C=2 ** 40), "R and C"), (dict(workspace=None), "workspace"), (dict(workspace=FAKE + 128), "workspace"), (dict(nbytes=ROOM - 1), "too small"),
    (dict(nbytes=-1), "too small"),
]


@pytest.mark.parametrize("kw,says", MATRICES + [(dict(x=None), "NULL"), (dict(out=None), "NULL"), (dict(x=FAKE + 2), "aligned"), (dict(out=FAKE + 1), "aligned"),
                                                (dict(dt=3), "type"), (dict(odt=-1), "type")])
def test_orthogonalize(kw, says):
    c = iteration()
    refused(call("mxq_orthogonalize", ORTHOGONALIZE | dict(cfg=ctypes.byref(c)), kw), says)


@pytest.mark.parametrize("kw,says", CONFIGS)
def test_iterations(kw, says):
    c = iteration(**kw)
    refused(call("mxq_orthogonalize", ORTHOGONALIZE, dict(cfg=ctypes.byref(c))), says)
    s = mxq.MuonConfig(c, 1e-3, 0.9, 0.1, 1.0, 1.0, 1)
    refused(call("mxq_muon", MUON, dict(cfg=ctypes.byref(s))), says)


def test_iterations_without_a_config():
    refused(call("mxq_orthogonalize", ORTHOGONALIZE, {}), "config")
    refused(call("mxq_muon", MUON, {}), "config")


MUON = dict(param=FAKE, param_dt=1, grad=FAKE, grad_dt=0, m=FAKE, copy=None, batch=2, R=40, C=50, cfg=None, control=None, workspace=FAKE, nbytes=ROOM,
            st=None)


@pytest.mark.parametrize("kw,says", MATRICES + [
    (dict(param=None), "NULL"), (dict(grad=None), "NULL"), (dict(m=None), "NULL"), (dict(param=FAKE + 1), "aligned"), (dict(grad=FAKE + 2), "aligned"),
    (dict(m=FAKE + 2), "aligned"), (dict(copy=FAKE + 1), "aligned"), (dict(control=FAKE + 8), "control"), (dict(param_dt=2), "type"),
    (dict(grad_dt=2), "type"), (dict(param_dt=0), "too small"),  # (fp32 results need more room)
])
def test_muon(kw, says):
    c = mxq.MuonConfig(iteration(), 1e-3, 0.9, 0.1, 1.0, 1.0, 1)
    refused(call("mxq_muon", MUON | dict(cfg=ctypes.byref(c)), kw), says)


@pytest.mark.parametrize("kw,says", [
    (dict(momentum=-0.1), "momentum"), (dict(momentum=1.0), "momentum"), (dict(momentum=NAN), "momentum"), (dict(nesterov=2), "nesterov"),
    (dict(nesterov=-1), "nesterov"), (dict(weight_decay=NAN), "weight_decay"), (dict(weight_decay=1e300), "weight_decay"), (dict(scale=INF), "scale"),
    (dict(scale=-1e39), "scale"),
])
def test_muon_config(kw, says):
    c = mxq.MuonConfig(iteration(), 1e-3, 0.9, 0.1, 1.0, 1.0, 1)
    for k, v in kw.items():
        setattr(c, k, v)
    refused(call("mxq_muon", MUON, dict(cfg=ctypes.byref(c))), says)


def test_workspace():
    of = mxq.mxq_orthogonalize_workspace
    for bad in ((-1, 4, 4, 0), (65536, 4, 4, 0), (1, 0, 4, 0), (1, 4, 2 ** 20 + 1, 0), (1, 4, 4, 2), (1, 4, 4, -1)):
        assert of(*bad) == 0
    for batch, R, C in ((1, 1, 1), (3, 70, 40), (4, 40, 70), (2, 4096, 7168)):
        lo, hi = (-(-min(R, C) // 64) * 64, -(-max(R, C) // 64) * 64)
        for dt, halves in ((1, 3 * lo * hi + 2 * lo * lo), (0, 2 * (2 * lo * hi + 2 * lo * lo))):
            assert 0 <= of(batch, R, C, dt) - batch * (2 * halves + 2048) < 6 * 256
        assert of(batch, R, C, 0) == of(batch, C, R, 0)
    assert 0 <= of(0, 5, 5, 0) < 6 * 256
    assert of(65535, 2 ** 20, 2 ** 20, 1) == 0 or of(65535, 2 ** 20, 2 ** 20, 1) > 2 ** 40  # never a wrapped size


@pytest.mark.skipif(HAS_GPU, reason="a GPU is present; this checks the no-device path")
def test_well_formed_calls_stop_at_the_device_gate():
    c = iteration()
    s = mxq.MuonConfig(c, 1e-3, 0.9, 0.1, 1.0, 1.0, 1)
    none = dict(x=None, q_row=None, s_row=None, q_colT=None, s_colT=None)
    assert call("mxq_quantize128", QUANTIZE, {}) == DEVICE and call("mxq_quantize128", QUANTIZE, none | dict(R=0)) == DEVICE
    assert call("mxq_quantize128", QUANTIZE, none | dict(batch=0)) == DEVICE
    assert call("mxq_quantize128", QUANTIZE, dict(axis_mask=1, q_colT=None, s_colT=None)) == DEVICE
    assert call("mxq_quantize128_grouped", GROUPED, {}) == DEVICE
    assert call("mxq_quantize128_grouped", GROUPED, dict(axis_mask=1, ldq=0, q_colT=None, s_colT=None)) == DEVICE
    assert call("mxq_gemm128", GEMM, {}) == DEVICE and call("mxq_gemm128", GEMM, dict(M=0, A=None, sA=None, C=None)) == DEVICE
    for mode in (0, 1):
        assert call("mxq_grouped_gemm128", GROUPED_GEMM, dict(mode=mode)) == DEVICE
    assert call("mxq_orthogonalize", ORTHOGONALIZE, dict(cfg=ctypes.byref(c))) == DEVICE
    assert call("mxq_orthogonalize", ORTHOGONALIZE, dict(cfg=ctypes.byref(c), batch=0, x=None, out=None, workspace=None, nbytes=0)) == DEVICE
    assert call("mxq_muon", MUON, dict(cfg=ctypes.byref(s))) == DEVICE
    for good in ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (0.0, 0.0, 0.0)):
        g = iteration(a=good[0], b=good[1], c=good[2])
        assert call("mxq_orthogonalize", ORTHOGONALIZE, dict(cfg=ctypes.byref(g))) == DEVICE


def test_struct_sizes_match_the_header(tmp_path):
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs the HIP headers")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = (("mxq_newton_schulz", mxq.NewtonSchulz), ("mxq_muon_config", mxq.MuonConfig))
    lines = [f'printf("{n} %zu %zu\\n", sizeof({n}), offsetof({n}, {f[0]}));' for n, c in pairs for f in c._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mxq.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(root, "include"), "-I/opt/rocm/include", str(src), "-o", exe], check=True)
    got = re.findall(r"mxq_\w+ (\d+) (\d+)", subprocess.run([exe], capture_output=True, text=True, check=True).stdout)
    assert got == [(str(ctypes.sizeof(c)), str(getattr(c, f[0]).offset)) for _, c in pairs for f in c._fields_]


# ---- the binding, with a tensor type that passes for a device tensor
class Dev(torch.Tensor):
    is_cuda = True

    @property
    def device_index(self):
        return getattr(self, "_index", 0)

    def get_device(self):
        return self.device_index


def dev(*shape, dtype=torch.float32, index=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Dev)
    t._index = index
    return t


U8, BF16, I32 = torch.uint8, torch.bfloat16, torch.int32


@pytest.fixture
def library(monkeypatch):
    """Entry points that note their calls and succeed, on a current device 0."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: 4096 if name in ("mxq_orthogonalize_workspace", "mxq_grouped128_cols_max") else calls.append(name) or 0

    monkeypatch.setattr(mxq, "_lib", Library())
    monkeypatch.setattr(mxq, "_device_count", lambda: 2)
    monkeypatch.setattr(mxq, "_current_device", lambda: 0)
    monkeypatch.setattr(mxq, "_current_stream", lambda index: 0)
    mxq.mxq_orthogonalize_workspace.cache_clear()
    yield calls
    mxq.mxq_orthogonalize_workspace.cache_clear()


def codes(rows, K, tile=1, lead=(), index=0):
    return dev(*lead, rows, K, dtype=U8, index=index), dev(*lead, K // 128, -(-rows // tile), index=index)


A, SA = codes(5, 256)
B, SB = codes(300, 256, 128)
W, SW = codes(300, 256, 128, (2,))
KB, SKB = codes(300, 256)
ENDS = dev(2, dtype=I32)
MISUSE = {
    "host tensor": (lambda: mxq.quantize128(torch.zeros(4, 4)), ValueError, "device tensor"),
    "half": (lambda: mxq.quantize128(dev(4, 4, dtype=torch.half)), TypeError, "float32 or bfloat16"),
    "four dims": (lambda: mxq.mxq_quantize128(dev(2, 2, 4, 4), 1, 1), ValueError, "2 dims"),
    "transposed": (lambda: mxq.quantize128(dev(8, 4).T), ValueError, "unit stride"),
    "tile": (lambda: mxq.quantize128(dev(4, 4), tile=2), ValueError, "tile"),
    "no outputs": (lambda: mxq.mxq_quantize128(dev(4, 4), 1, 1), TypeError, "q_row"),
    "narrow codes": (lambda: mxq.mxq_quantize128(dev(4, 200), 1, 1, dev(4, 200, dtype=U8), dev(2, 4)), ValueError, "q_row"),
    "scales by rows": (lambda: mxq.mxq_quantize128(dev(4, 200), 1, 1, dev(4, 256, dtype=U8), dev(4, 2)), ValueError, "s_row"),
    "scales of tiles": (lambda: mxq.mxq_quantize128(dev(4, 200), 128, 1, dev(4, 256, dtype=U8), dev(2, 4)), ValueError, "s_row"),
    "group ends' type": (lambda: mxq.quantize128_grouped(dev(4, 4), dev(2)), TypeError, "group_end"),
    "group ends apart": (lambda: mxq.quantize128_grouped(dev(4, 4), dev(4, dtype=I32)[::2]), ValueError, "group_end"),
    "codes' type": (lambda: mxq.gemm128(dev(5, 256), SA, B, SB), TypeError, "A must be"),
    "scales' shape": (lambda: mxq.gemm128(A, dev(5, 2), B, SB), ValueError, "sA must"),
    "no scales": (lambda: mxq.gemm128(A, None, B, SB), TypeError, "sA"),
    "other K": (lambda: mxq.gemm128(A, SA, *codes(300, 384, 128)), ValueError, "disagree"),
    "codes apart": (lambda: mxq.gemm128(dev(5, 512, dtype=U8)[:, ::2], SA, B, SB), ValueError, "contiguous"),
    "output's type": (lambda: mxq.gemm128(A, SA, B, SB, dtype=torch.half), TypeError, "float"),
    "output's shape": (lambda: mxq.mxq_gemm128(A, SA, B, SB, dev(300, 5)), ValueError, "C must"),
    "experts": (lambda: mxq.grouped_gemm128(0, A, SA, *codes(300, 256, 128, (3,)), ENDS), ValueError, "B must"),
    "experts by rows": (lambda: mxq.grouped_gemm128(0, A, SA, *codes(300, 256, 1, (2,)), ENDS), ValueError, "sB must"),
    "tiles along tokens": (lambda: mxq.grouped_gemm128(1, A, SA, B, SB, ENDS), ValueError, "sB must"),
    "grouped output": (lambda: mxq.mxq_grouped_gemm128(1, A, SA, KB, SKB, dev(5, 300), ENDS), ValueError, "C must"),
    "matrix apart": (lambda: mxq.orthogonalize(dev(4, 8)[:, ::2]), ValueError, "contiguous"),
    "one dim": (lambda: mxq.orthogonalize(dev(4)), ValueError, "2 or 3 dims"),
    "result's type": (lambda: mxq.orthogonalize(dev(4, 4), dtype=torch.half), TypeError, "float"),
    "result's shape": (lambda: mxq.mxq_orthogonalize(dev(4, 4), mxq.newton_schulz(), dev(4, 5), dev(9, dtype=U8)), ValueError, "out must"),
    "lengths": (lambda: mxq.Muon([dev(4, 4)], [], []), ValueError, "one length"),
    "gradient's shape": (lambda: mxq.Muon([dev(4, 4)], [dev(16, 1)], [dev(4, 4)]), ValueError, "grad must"),
    "momentum's type": (lambda: mxq.Muon([dev(4, 4)], [dev(4, 4)], [dev(4, 4, dtype=BF16)]), TypeError, "m must"),
    "copy's type": (lambda: mxq.Muon([dev(4, 4)], [dev(4, 4)], [dev(4, 4)], [dev(4, 4)]), TypeError, "copy must"),
    "rule": (lambda: mxq.muon_scale((4, 4), "none"), ValueError, "rule"),
    "control": (lambda: mxq.Muon([dev(4, 4)], [dev(4, 4)], [dev(4, 4)]).step(control=dev(4)), TypeError, "control"),
    # another device than the current one, or two devices
    "x elsewhere": (lambda: mxq.quantize128(dev(4, 4, index=1)), ValueError, "current device"),
    "ends elsewhere": (lambda: mxq.quantize128_grouped(dev(4, 4), dev(2, dtype=I32, index=1)), ValueError, "another tensor"),
    "weights elsewhere": (lambda: mxq.gemm128(A, SA, *codes(300, 256, 128, index=1)), ValueError, "another tensor"),
    "experts elsewhere": (lambda: mxq.grouped_gemm128(0, A, SA, *codes(300, 256, 128, (2,), 1), ENDS), ValueError, "another tensor"),
    "matrix elsewhere": (lambda: mxq.mxq_orthogonalize(dev(4, 4, index=1), mxq.newton_schulz(), dev(4, 4, index=1), dev(9, dtype=U8, index=1)), ValueError, "current device"),
    "gradient elsewhere": (lambda: mxq.mxq_muon(dev(4, 4), dev(4, 4, index=1), dev(4, 4), mxq.MuonConfig(), dev(9, dtype=U8)), ValueError, "another tensor"),
}


@pytest.mark.parametrize("name", MISUSE)
def test_the_binding_refuses(name, library):
    f, error, says = MISUSE[name]
    with pytest.raises(error, match=says):
        f()
    assert not library


CALLS = {
    "quantize128": lambda st: mxq.quantize128(dev(140, 200), 3, stream=st),
    "quantize128 of tiles": lambda st: mxq.quantize128(dev(2, 140, 200, dtype=BF16), 3, 128, stream=st),
    "quantize128_grouped": lambda st: mxq.quantize128_grouped(dev(140, 200), ENDS, 3, stream=st),
    "gemm128": lambda st: mxq.gemm128(A, SA, B, SB, stream=st),
    "gemm128 of rows": lambda st: mxq.gemm128(A, SA, KB, SKB, torch.float32, stream=st),
    "grouped_gemm128 ragged M": lambda st: mxq.grouped_gemm128(0, A, SA, W, SW, ENDS, stream=st),
    "grouped_gemm128 ragged K": lambda st: mxq.grouped_gemm128(1, A, SA, KB, SKB, ENDS, stream=st),
    "orthogonalize": lambda st: mxq.orthogonalize(dev(3, 40, 50), stream=st),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_helpers_memory_is_its_streams(name, library, monkeypatch):
    """Outputs and temporaries are allocated, and the call runs, within the stream that is given."""
    events = []

    @contextlib.contextmanager
    def on(stream, device):
        events.append("within")
        yield
        events.append("left")

    def noting(of):
        def made(*a, **kw):
            events.append("made")
            return of(*a, **kw).as_subclass(Dev)
        return made

    monkeypatch.setattr(mxq, "_on", on)
    for owner, func in ((torch, "empty"), (torch, "empty_like"), (Dev, "new_empty")):
        monkeypatch.setattr(owner, func, noting(getattr(owner, func)), raising=False)
    CALLS[name](5)
    assert len(library) == 1 and events[0] == "within" and events[-1] == "left" and events.count("within") == 1 and "made" in events
    events.clear()
    CALLS[name](None)
    assert len(library) == 2 and "within" not in events and "made" in events


def test_update_sizes():
    assert mxq.muon_scale((4, 100, 400)) == pytest.approx(0.2 * 20)
    assert mxq.muon_scale((400, 100), "original") == 2 and mxq.muon_scale((100, 400), "original") == 1
    assert math.isclose(mxq.muon_scale((1, 1)), 0.2)
