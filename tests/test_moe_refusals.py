"""Arguments that the router, combine and AdamW entry points refuse, on the host: no GPU is reached."""
import ctypes
import os

import pytest
import torch

from moe_grouped_gemm_mxq_amd import mxq

INVALID, DEVICE = 1, 3
FAKE, ODD = 0x10000, 0x10001  # never dereferenced: the checks end first
HAS_GPU = torch.cuda.device_count() > 0


def last():
    return mxq.mxq_last_error()


def cfg(**kw):
    c = mxq.RouteConfig(0, 2, 1, 1, 1, 1, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def route(c=None, **kw):
    a = dict(logits=FAKE, dt=0, T=4, E=16, ld=16, bias=None, cfg=ctypes.byref(cfg() if c is None else c), idx=FAKE, weights=FAKE,
             group_end=None, row_token=None, slot=None, workspace=None, nbytes=0, st=None)
    a.update(kw)
    return mxq._lib.mxq_route(*a.values())


BIG = mxq.mxq_expert_order_workspace(4, 2, 16)


@pytest.mark.parametrize("kw,says", [
    (dict(logits=None), "NULL"), (dict(logits=ODD), "aligned"), (dict(logits=FAKE + 2), "aligned"), (dict(dt=2), "type"),
    (dict(dt=-1), "type"), (dict(T=-1), "T must"), (dict(E=0), "E must"), (dict(E=1025), "E must"), (dict(ld=15), "stride"),
    (dict(idx=None), "NULL"), (dict(weights=None), "NULL"), (dict(idx=ODD), "aligned"), (dict(weights=FAKE + 2), "aligned"),
    (dict(bias=FAKE + 2), "aligned"), (dict(cfg=None), "config"), (dict(T=2 ** 31), "2^31"),
    (dict(group_end=FAKE), "NULL"), (dict(slot=FAKE), "NULL"),
    (dict(group_end=FAKE, row_token=FAKE, slot=FAKE), "workspace"),
    (dict(group_end=FAKE, row_token=FAKE, slot=FAKE, workspace=FAKE, nbytes=BIG - 1), "workspace"),
    (dict(group_end=FAKE, row_token=FAKE, slot=FAKE, workspace=FAKE + 8, nbytes=BIG), "aligned"),
    (dict(group_end=FAKE, row_token=FAKE, slot=FAKE + 2, workspace=FAKE, nbytes=BIG), "aligned"),
])
def test_route(kw, says):
    assert route(**kw) == INVALID
    assert says in last()


@pytest.mark.parametrize("kw,says", [
    (dict(score=2), "score"), (dict(score=-1), "score"), (dict(top_k=0), "top_k"), (dict(top_k=17), "top_k"),
    (dict(n_group=0), "n_group"), (dict(n_group=3), "n_group"), (dict(topk_group=2), "topk_group"), (dict(topk_group=0), "topk_group"),
    (dict(group_top=0), "group_top"), (dict(group_top=3), "group_top"), (dict(renormalise=2), "renormalise"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
])
def test_route_config(kw, says):
    assert route(cfg(**kw)) == INVALID
    assert says in last()


def test_limits_of_top_k_and_groups():
    assert route(cfg(top_k=33), E=64, ld=64) == INVALID and "top_k" in last()
    assert route(cfg(n_group=128), E=1024, ld=1024) == INVALID and "n_group" in last()


@pytest.mark.parametrize("kw,says", [(dict(ldd=15), "stride"), (dict(dlogits=None), "NULL"), (dict(dlogits=FAKE + 2), "aligned"),
                                     (dict(idx=None), "NULL"), (dict(dweights=None), "NULL"), (dict(dweights=ODD), "aligned"),
                                     (dict(logits=None), "NULL"), (dict(T=-1), "T must"), (dict(ld=3), "stride")])
def test_route_backward(kw, says):
    a = dict(logits=FAKE, dt=0, T=4, E=16, ld=16, cfg=ctypes.byref(cfg()), idx=FAKE, dweights=FAKE, dlogits=FAKE, ldd=16, st=None)
    a.update(kw)
    assert mxq._lib.mxq_route_backward(*a.values()) == INVALID
    assert says in last()


@pytest.mark.parametrize("kw,says", [(dict(idx=None), "NULL"), (dict(idx=ODD), "aligned"), (dict(T=-1), "T must"), (dict(K=0), "top_k"),
                                     (dict(K=33), "top_k"), (dict(E=0), "E must"), (dict(E=1025), "E must"), (dict(ge=None), "NULL"),
                                     (dict(tok=None), "NULL"), (dict(slot=None), "NULL"), (dict(ws=None), "workspace"),
                                     (dict(n=BIG - 4), "workspace"), (dict(ws=FAKE + 4), "aligned"), (dict(T=2 ** 31), "2^31")])
def test_expert_order(kw, says):
    a = dict(idx=FAKE, T=4, K=2, E=16, ge=FAKE, tok=FAKE, slot=FAKE, ws=FAKE, n=BIG, st=None)
    a.update(kw)
    assert mxq._lib.mxq_expert_order(*a.values()) == INVALID
    assert says in last()


def test_workspace_of_refused_arguments_is_zero():
    for a in ((-1, 2, 16), (4, 0, 16), (4, 33, 64), (4, 2, 0), (4, 2, 1025), (2 ** 31, 1, 4), (2 ** 30, 2, 4)):
        assert mxq.mxq_expert_order_workspace(*a) == 0
    assert BIG > 0 and mxq.mxq_expert_order_workspace(0, 1, 1) > 0


COMBINE = dict(y=FAKE, ydt=0, rows=8, ldy=16, slot=FAKE, weights=FAKE, T=4, K=2, H=16, out=FAKE, odt=1, ldo=16, st=None)


@pytest.mark.parametrize("kw,says", [(dict(y=None), "NULL"), (dict(y=FAKE + 2), "aligned"), (dict(ydt=2), "type"), (dict(odt=-1), "type"),
                                     (dict(rows=-1), "rows"), (dict(rows=2 ** 31), "rows"), (dict(ldy=15), "stride"), (dict(ldo=15), "stride"),
                                     (dict(slot=None), "NULL"), (dict(slot=FAKE + 2), "aligned"), (dict(weights=ODD), "aligned"),
                                     (dict(T=-1), "T must"), (dict(T=2 ** 31), "T must"), (dict(K=0), "top_k"), (dict(K=33), "top_k"),
                                     (dict(H=0), "H must"), (dict(out=None), "NULL"), (dict(out=ODD), "aligned")])
def test_combine(kw, says):
    assert mxq._lib.mxq_combine(*{**COMBINE, **kw}.values()) == INVALID
    assert says in last()


@pytest.mark.parametrize("kw,says", [(dict(dout=None), "NULL"), (dict(dout=FAKE + 2), "aligned"), (dict(dt=7), "type"), (dict(ldd=1), "stride"),
                                     (dict(y=None), "NULL"), (dict(ldy=8), "stride"), (dict(ydt=3), "type"), (dict(dydt=3), "type"),
                                     (dict(lddy=8), "stride"), (dict(dy=ODD), "aligned"), (dict(dw=FAKE + 2), "aligned"),
                                     (dict(rows=-1), "rows"), (dict(H=-4), "H must"), (dict(K=40), "top_k"), (dict(slot=None), "NULL")])
def test_combine_backward(kw, says):
    a = dict(dout=FAKE, dt=0, ldd=16, y=FAKE, ydt=0, ldy=16, slot=FAKE, weights=FAKE, T=4, K=2, H=16, rows=8, dy=FAKE, dydt=0, lddy=16,
             dw=FAKE, st=None)
    a.update(kw)
    assert mxq._lib.mxq_combine_backward(*a.values()) == INVALID
    assert says in last()


def adamw(tensor=None, config=None, n=1, pdt=0, gdt=0, fmt=0, control=None, array=True):
    t = (mxq.AdamWTensor * 2)()
    for k, v in {**dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, n=100, decay_scale=1.0), **(tensor or {})}.items():
        setattr(t[0], k, v)
    c = mxq.AdamWConfig(1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, 0)
    for k, v in (config or {}).items():
        setattr(c, k, v)
    return mxq._lib.mxq_adamw(t if array else None, n, pdt, gdt, fmt, None if config is False else ctypes.byref(c), control, None)


@pytest.mark.parametrize("kw,says", [
    (dict(n=-1), "n_tensors"), (dict(array=False), "NULL"), (dict(pdt=2), "parameter type"), (dict(gdt=2), "gradient type"),
    (dict(fmt=2), "state format"), (dict(config=False), "config"), (dict(control=FAKE + 4), "control"),
    (dict(config=dict(beta1=1.0)), "betas"), (dict(config=dict(beta2=-0.1)), "betas"), (dict(config=dict(beta2=float("nan"))), "betas"),
    (dict(config=dict(eps=0.0)), "eps"), (dict(config=dict(eps=float("nan"))), "eps"), (dict(config=dict(lr=float("inf"))), "lr"),
    (dict(config=dict(weight_decay=float("nan"))), "weight_decay"), (dict(config=dict(step=0)), "step"),
    (dict(tensor=dict(n=-1)), "n must"), (dict(tensor=dict(param=None)), "NULL"), (dict(tensor=dict(grad=None)), "NULL"),
    (dict(tensor=dict(m=None)), "NULL"), (dict(tensor=dict(v=None)), "NULL"), (dict(tensor=dict(decay_scale=float("nan"))), "decay_scale"),
    (dict(tensor=dict(param=FAKE + 2)), "aligned"), (dict(tensor=dict(grad=ODD), gdt=1), "aligned"), (dict(tensor=dict(m=FAKE + 1)), "aligned"),
    (dict(tensor=dict(copy=ODD)), "aligned"), (dict(fmt=1), "m_scale"), (dict(fmt=1, tensor=dict(m_scale=FAKE)), "v_scale"),
    (dict(tensor=dict(n=2 ** 40)), "too many"),
])
def test_adamw(kw, says):
    assert adamw(**kw) == INVALID
    assert says in last()


@pytest.mark.skipif(HAS_GPU, reason="a GPU is present; this checks the no-device path")
def test_well_formed_calls_stop_at_the_device_gate():
    assert route() == DEVICE and last()
    assert mxq._lib.mxq_combine(*COMBINE.values()) == DEVICE
    assert adamw() == DEVICE and adamw(n=0) == DEVICE
    assert adamw(fmt=1, tensor=dict(m_scale=ODD, v_scale=ODD, m=ODD, v=ODD, copy=FAKE + 2)) == DEVICE


def test_the_binding_refuses_wrong_tensors():
    """Host tensors, types and shapes; a meta tensor stands for one of the wrong kind."""
    x = torch.randn(4, 16)
    with pytest.raises(ValueError, match="device tensor"):
        mxq.route(x, 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mxq.route(x.half(), 2)
    with pytest.raises(ValueError, match="score"):
        mxq.route(x, 2, score="tanh")
    with pytest.raises(ValueError, match="device tensor"):
        mxq.combine(x, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="torch.Tensor"):
        mxq.mxq_combine(None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        mxq.AdamW([x], [x], [x], [x])
    with pytest.raises(ValueError, match="one length"):
        mxq.AdamW([x], [x], [x], [])
    with pytest.raises(TypeError, match="param must be"):
        mxq.AdamW([x.half()], [x], [x], [x])


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structures are the header's, field by field."""
    import re
    import subprocess
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs the HIP headers")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = (("mxq_route_config", mxq.RouteConfig), ("mxq_adamw_tensor", mxq.AdamWTensor), ("mxq_adamw_config", mxq.AdamWConfig))
    lines = [f'printf("{n} %zu %zu\\n", sizeof({n}), offsetof({n}, {f[0]}));' for n, c in pairs for f in c._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mxq.h"\nint main(void) {' + "\n".join(lines)
                   + 'printf("control %zu\\n", sizeof(mxq_adamw_control)); return 0; }')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(root, "include"), "-I/opt/rocm/include", str(src), "-o", exe], check=True)
    got = re.findall(r"mxq_\w+ (\d+) (\d+)", subprocess.run([exe], capture_output=True, text=True, check=True).stdout)
    want = [(str(ctypes.sizeof(c)), str(getattr(c, f[0]).offset)) for _, c in pairs for f in c._fields_]
    assert got == want


@pytest.mark.parametrize("eps", [1e-300, 1e-46, 2.0 ** -149, 1e-39, 2.0 ** -127, -1e-8, float("inf")])
def test_adamw_eps_has_to_be_normal_in_fp32(eps):
    """An eps that fp32 has as 0 or as a subnormal would turn elements without gradient or state into NaN."""
    assert adamw(config=dict(eps=eps)) == INVALID and "eps" in last()
    assert adamw(config=dict(eps=2.0 ** -126), tensor=dict(param=None)) == INVALID and "NULL" in last()  # accepted: the next check ends it
