"""Cases of the operators around the expert GEMMs of an MoE training step: the router with its expert order
and gradient, the weighted combine of the experts' rows with its gradient, and the AdamW step of many tensors.

``run`` computes a case in its plain form (elementary torch operations) or, where ``own`` is true, through the
library's entry points, on the inputs that ``prepare`` makes; ``exact`` gives the same outputs from the
operators' definitions in 64 bits; ``work`` gives the bytes and operations a pass cannot do without.

Definitions
  route     score s = softmax(l) or sigmoid(l) over E experts; key = s + bias, or the logit where there is no
            bias; of n_group equal groups those topk_group stay whose sums of the best `group_top` s (+ bias)
            are largest; the top_k largest keys, ties to the lowest index; weight scale * s, or scale * s / (sum
            of the chosen s).  A logit at or below the lowest finite bf16 value masks its expert: it is never
            chosen, and a row with too few experts ends in index -1 and weight 0.  Expert order: the (token, k)
            pairs sorted stably by expert give each pair's row (`slot`), each row's token and the group ends.
  combine   out[t] = sum_k w[t, k] y[slot[t, k]] over the slots >= 0.
  adamw     g' = grad_scale g; m' = b1 m + (1 - b1) g'; v' = b2 v + (1 - b2) g'^2;
            p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
            8-bit states: E4M3 elements of m and of r = sqrt(v) in blocks of 32 with one power-of-two scale, the
            smallest that keeps the block's largest finite magnitude at or below 448, rounded stochastically:
            y -> step * floor(y / step + u), u in (0, 1) from a counter hash of (seed, step, tensor, element);
            a positive r does not round to 0.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
LOWEST = -3.3895313892515355e38  # lowest finite bf16 value: logits at or below it are masked
MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a small batch: grouped sigmoid routing with a balance bias; latency counts
        {"name": "route_decode", "op": "route", "T": 7, "E": 256, "K": 8, "score": "sigmoid", "bias": True, "n_group": 8,
         "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "fp32", "masked": False},
        # a training step's tokens over 256 experts in 8 groups
        {"name": "route_train_grouped", "op": "route", "T": 16384, "E": 256, "K": 8, "score": "sigmoid", "bias": True,
         "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "fp32", "masked": False},
        # the 32 local experts of the MoE layer, bf16 logits of a ragged token count, some experts masked off
        {"name": "route_experts32", "op": "route", "T": 5003, "E": 32, "K": 8, "score": "softmax", "bias": False, "n_group": 1,
         "topk_group": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "bf16", "masked": True},
        # gradient of plain softmax weights: every logit of the row takes part
        {"name": "route_backward_softmax", "op": "route_backward", "T": 16384, "E": 256, "K": 8, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "fp32", "masked": False},
        # gradient of renormalised sigmoid weights on a small odd batch
        {"name": "route_backward_sigmoid", "op": "route_backward", "T": 61, "E": 96, "K": 6, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "dtype": "bf16", "masked": False},
        # decoding: a few tokens' bf16 expert rows
        {"name": "combine_decode", "op": "combine", "T": 7, "K": 8, "H": 7168, "y": "bf16", "out": "bf16", "weights": True,
         "dropped": False},
        # the MoE layer's routed rows as the ragged-M GEMM leaves them
        {"name": "combine_train", "op": "combine", "T": 16384, "K": 8, "H": 4096, "y": "fp32", "out": "bf16", "weights": True,
         "dropped": False},
        # its gradient: the rows' gradients in expert order, for the quantiser, and the router weights' gradients
        {"name": "combine_backward_train", "op": "combine_backward", "T": 16384, "K": 8, "H": 4096, "y": "fp32", "out": "bf16",
         "weights": True, "dropped": False},
        # odd sizes, and slots dropped by a capacity limit
        {"name": "combine_backward_odd", "op": "combine_backward", "T": 1003, "K": 3, "H": 1237, "y": "bf16", "out": "bf16",
         "weights": True, "dropped": True},
        # the small tensors of a layer (norms, biases, router rows), 32-bit states
        {"name": "adamw_small", "op": "adamw", "tensors": 48, "total": 120000, "ragged": True, "packed": False, "param": "fp32",
         "grad": "fp32", "bits": 32, "copy": False},
        # weights in bf16 with bf16 gradients, 32-bit states
        {"name": "adamw_weights_32", "op": "adamw", "tensors": 5, "total": 5 * 7168 * 4096, "ragged": False, "packed": False,
         "param": "bf16", "grad": "bf16", "bits": 32, "copy": False},
        # the 32 experts' weight tensor: fp32 with the bf16 copy that the quantiser reads, the weight-gradient GEMM's fp32 output, 8-bit states
        {"name": "adamw_experts_8", "op": "adamw", "tensors": 1, "total": 32 * 7168 * 4096, "ragged": False, "packed": False,
         "param": "fp32", "grad": "fp32", "bits": 8, "copy": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["route", "route", "route_backward", "combine", "combine_backward", "adamw", "adamw"])
    coin = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("route", "route_backward"):
        n_group = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        per = _log(rng, 8, 512 // n_group)
        E = n_group * per
        K = rng.randint(1, 8)
        need = -(-K // per)
        c = {"op": op, "T": min(_log(rng, 1, 16384), 16384 * 256 // E), "E": E, "K": K, "score": rng.choice(["softmax", "sigmoid"]),
             "renorm": coin(), "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["fp32", "bf16"]), "masked": coin(0.3)}
        if op == "route":
            c |= {"bias": coin(), "n_group": n_group, "topk_group": rng.randint(need, n_group), "group_top": rng.choice([1, 2])}
        return c
    if op in ("combine", "combine_backward"):
        K, H = rng.randint(1, 8), _log(rng, 64, 7168)
        return {"op": op, "T": min(_log(rng, 1, 16384), 16384 * 8 * 4096 // (K * H)), "K": K, "H": H, "y": rng.choice(["fp32", "bf16"]),
                "out": rng.choice(["fp32", "bf16"]), "weights": coin(0.8), "dropped": coin(0.3)}
    param = rng.choice(["fp32", "bf16"])
    return {"op": op, "tensors": _log(rng, 1, 64), "total": _log(rng, 1000, 2e8), "ragged": coin(), "packed": coin(0.3), "param": param,
            "grad": rng.choice(["fp32", "bf16"]), "bits": rng.choice([8, 32]), "copy": param == "fp32" and coin()}


# ------------------------------------------------------------------ inputs
def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _sizes(case):
    """Element counts of an AdamW case's tensors: equal ones, or odd ones of a wide spread."""
    n, total = case["tensors"], case["total"]
    if not case["ragged"]:
        return [max(1, total // n)] * n
    w = [((j + 1) * 0.6180339887498949 % 1.0) ** 4 + 1e-3 for j in range(n)]
    return [max(1, int(total * x / sum(w)) | 1) for x in w]


def _spans(sizes, gap):
    at, spans = 0, []
    for n in sizes:
        spans.append((at, n))
        at = -(-(at + n) // gap) * gap
    return spans, at


def _dropped(case):
    pairs = case["T"] * case["K"]
    return min(pairs, case["K"] + pairs // 5) if case["dropped"] else 0


def _logits(case, g):
    x = (1.5 * torch.randn(case["T"], case["E"], generator=g, device=DEV)).to(_dt(case["dtype"]))
    if case["masked"]:  # a tenth of the experts unavailable, and one row with none at all
        x[torch.rand(x.shape, generator=g, device=DEV) < 0.1] = -math.inf
        x[case["T"] // 2] = torch.finfo(x.dtype).min
    return x


def _encode_nearest(x):
    """E4M3 elements and E8M0 scales of a flat fp32 tensor in blocks of 32, rounded to nearest."""
    b = torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 32)
    e = torch.clamp(torch.ceil(torch.log2(b.abs().amax(1, keepdim=True) / 448.0)), -126, 127)
    code = (b * torch.exp2(-e)).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[: x.numel()]
    return code.clone(), (e + 127).to(torch.uint8).view(-1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = _logits(case, g)
        if op == "route":
            s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
            i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=DEV)  # noqa: E731
            s["out"] = {"idx": i32(T, K), "weights": torch.empty(T, K, device=DEV), "group_end": i32(E), "row_token": i32(T * K),
                        "slot": i32(T, K)}
        else:
            top, idx = torch.topk(s["logits"].float(), K, dim=1)
            s["idx"] = torch.where(top <= LOWEST, -1, idx).to(torch.int32)
            s["dweights"] = torch.randn(T, K, generator=g, device=DEV)
        return s
    if op in ("combine", "combine_backward"):
        T, K, H = case["T"], case["K"], case["H"]
        experts = max(K, 32)
        idx = torch.rand(T, experts, generator=g, device=DEV).topk(K, dim=1).indices.reshape(-1)
        if case["dropped"]:  # one token lost all of its experts, and a fifth of the pairs found no room
            chance = torch.rand(T, K, generator=g, device=DEV)
            chance[T // 2] = -1.0
            idx[torch.argsort(chance.view(-1))[: _dropped(case)]] = experts
        order = torch.argsort(idx, stable=True)
        slot = torch.empty_like(order)
        slot[order] = torch.arange(T * K, device=DEV)
        rows = T * K - _dropped(case)
        s["rows"] = rows
        s["slot"] = torch.where(slot < rows, slot, -1).to(torch.int32).view(T, K)
        s["weights"] = torch.rand(T, K, generator=g, device=DEV) if case["weights"] else None
        if op == "combine" or case["weights"]:
            s["y"] = torch.randn(rows, H, generator=g, device=DEV).to(_dt(case["y"]))
        if op == "combine_backward":
            s["dout"] = torch.randn(T, H, generator=g, device=DEV).to(_dt(case["out"]))
        return s
    sizes = _sizes(case)
    spans, flat = _spans(sizes, 1 if case["packed"] else 64)
    bspans, bflat = _spans([-(-n // 32) for n in sizes], 1)
    s["param"] = (0.02 * torch.randn(flat, generator=g, device=DEV)).to(_dt(case["param"]))
    s["grad"] = torch.randn(flat, generator=g, device=DEV).mul_(1e-3).to(_dt(case["grad"]))
    m = torch.randn(flat, generator=g, device=DEV).mul_(3e-4)
    v = torch.rand(flat, generator=g, device=DEV).add_(0.2).mul_(1e-6)
    if case["bits"] == 8:
        v.sqrt_()
        for name, x in (("m", m), ("v", v)):
            s[name], s[name + "_scale"] = torch.zeros(flat, dtype=torch.uint8, device=DEV), torch.zeros(bflat, dtype=torch.uint8, device=DEV)
            for (o, n), (bo, bn) in zip(spans, bspans):
                s[name][o:o + n], s[name + "_scale"][bo:bo + bn] = _encode_nearest(x[o:o + n])
    else:
        s["m"], s["v"] = m, v
    s["copy"] = torch.zeros(flat, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    s["spans"], s["bspans"] = spans, bspans
    s["hyper"] = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.01, "grad_scale": 0.5, "step": 100, "seed": seed & MASK32}
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from moe_grouped_gemm_mxq_amd import mxq

    c = s["case"]
    if c["op"] == "route":
        return mxq.route(s["logits"], c["K"], score=c["score"], bias=s["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
                         group_top=c["group_top"], renormalise=c["renorm"], scale=c["scale"], out=s["out"])
    if c["op"] == "route_backward":
        return mxq.route_backward(s["logits"], s["idx"], s["dweights"], score=c["score"], renormalise=c["renorm"], scale=c["scale"])
    if c["op"] == "combine":
        return mxq.combine(s["y"], s["slot"], s["weights"], dtype=_dt(c["out"]))
    if c["op"] == "combine_backward":
        dy, dw = mxq.combine_backward(s["dout"], s["slot"], s["rows"], weights=s["weights"], y=s.get("y"))
        return {"dy": dy, "dweights": dw}
    if "plan" not in s:  # a program makes it once, with its tensors
        cut = lambda x, spans: None if x is None else [x[o:o + n] for o, n in spans]  # noqa: E731
        m, v = cut(s["m"], s["spans"]), cut(s["v"], s["spans"])
        if c["bits"] == 8:
            m, v = list(zip(m, cut(s["m_scale"], s["bspans"]))), list(zip(v, cut(s["v_scale"], s["bspans"])))
        s["plan"] = mxq.AdamW(cut(s["param"], s["spans"]), cut(s["grad"], s["spans"]), m, v, copies=cut(s["copy"], s["spans"]))
    s["plan"].step(**s["hyper"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if s["case"]["bits"] == 8:  # element times scale is the state
        for name in ("m", "v"):
            out[name], out[name + "_scale"] = s[name].view(torch.float8_e4m3fn), s[name + "_scale"].view(torch.float8_e8m0fnu)
    return out


def _run_plain(s):
    return {"route": _route_plain, "route_backward": _route_backward_plain, "combine": _combine_plain,
            "combine_backward": _combine_backward_plain, "adamw": _adamw_plain}[s["case"]["op"]](s)


def _scores(x, kind):
    """Scores of logits x (masked ones -inf), in x's type."""
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return e / e.sum(1, keepdim=True).clamp_min(torch.finfo(x.dtype).tiny)


def _route_plain(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["n_group"]
    x = s["logits"].double()  # neighbouring keys of a row are compared: 64 bits
    masked = x <= LOWEST
    x = torch.where(masked, -math.inf, x)
    score = _scores(x, c["score"])
    biased = torch.where(masked, -math.inf, score if s["bias"] is None else score + s["bias"].double())
    key = x if s["bias"] is None else biased
    if G > 1:
        best = torch.sort(biased.view(T, G, E // G), dim=2, descending=True).values[:, :, : c["group_top"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(some, torch.where(best == -math.inf, 0.0, best).sum(2), -math.inf)
        groups = torch.sort(total, dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, groups, True)
        key = torch.where(kept[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    top, idx = top[:, :K], idx[:, :K]
    there = top > -math.inf
    w = torch.where(there, score.gather(1, idx), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float64).tiny)
    flat = torch.where(there, idx, E).reshape(-1)
    order = torch.argsort(flat, stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * K, device=x.device)
    ends = (flat[:, None] == torch.arange(E, device=x.device)).sum(0).cumsum(0)
    rows = torch.arange(T * K, device=x.device) < ends[-1]
    i32 = torch.int32
    return {"idx": torch.where(there, idx, -1).to(i32), "weights": (w * c["scale"]).float(), "group_end": ends.to(i32),
            "row_token": torch.where(rows, order // K, -1).to(i32), "slot": torch.where(there, slot.view(T, K), -1).to(i32)}


def _route_backward_plain(s):
    c = s["case"]
    x = s["logits"].float()
    x = torch.where(x <= LOWEST, -math.inf, x)
    there = s["idx"] >= 0
    idx = torch.where(there, s["idx"], 0).long()
    g = torch.where(there, s["dweights"], 0.0) * c["scale"]
    out = torch.zeros_like(x)
    if c["renorm"]:
        score = torch.where(there, _scores(x, c["score"]).gather(1, idx), 0.0)
        p = score / score.sum(1, keepdim=True).clamp_min(torch.finfo(x.dtype).tiny)
        d = p * (g - (p * g).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1.0 - score)
        out.scatter_add_(1, idx, torch.where(there, d, 0.0))
    elif c["score"] == "sigmoid":
        score = _scores(x, "sigmoid").gather(1, idx)
        out.scatter_add_(1, idx, torch.where(there, g * score * (1.0 - score), 0.0))
    else:
        score = _scores(x, "softmax")
        out.scatter_add_(1, idx, g)
        out = score * (out - (score * out).sum(1, keepdim=True))
    return out.to(s["logits"].dtype)


def _rows_of(s):
    there = (s["slot"] >= 0)
    w = there.float() if s["weights"] is None else torch.where(there, s["weights"], 0.0)
    return there, w


def _combine_plain(s):
    if not s["rows"]:
        return torch.zeros(s["slot"].shape[0], s["y"].shape[1], dtype=_dt(s["case"]["out"]), device=s["y"].device)
    there, w = _rows_of(s)
    rows = s["y"][torch.where(there, s["slot"], 0).long()].float()
    return (rows * w[:, :, None]).sum(1).to(_dt(s["case"]["out"]))


def _combine_backward_plain(s):
    there, w = _rows_of(s)
    T, K = s["slot"].shape
    d = s["dout"].float()
    dy = torch.zeros(s["rows"] + 1, d.shape[1], dtype=s["dout"].dtype, device=d.device)
    dy[torch.where(there, s["slot"], s["rows"]).long()] = (w[:, :, None] * d[:, None, :]).to(dy.dtype)
    dw = None
    if s["weights"] is not None:
        rows = s["y"][torch.where(there, s["slot"], 0).long()].float() if s["rows"] else torch.zeros(T, K, d.shape[1], device=d.device)
        dw = torch.where(there, (rows * d[:, None, :]).sum(2), 0.0)
    return {"dy": dy[: s["rows"]], "dweights": dw}


def _mix(x):
    x = (x ^ (x >> 16)) * 0x6A09E667 & MASK32
    x = (x ^ (x >> 15)) * 0xBB67AE85 & MASK32
    return x ^ (x >> 16)


def _uniforms(seed, step, tensor, n, device):
    """The hash's numbers in (0, 1) for the elements of m and of r of a tensor: one 64-bit product for two elements."""
    key = _mix((seed + 0x9E3779B9 * step + 0xBB67AE85 * (tensor + 1)) & MASK32)
    q = torch.arange((n + 1) // 2, device=device)
    x = (key + q * 0x9E3779B9 + (q >> 32) * 0x243F6A89) & MASK32
    x = (x ^ (x >> 15)) * 0x6A09E667 & MASK32
    x = (x ^ (x >> 13)) * 0xBB67AE85
    both = lambda even, odd: ((torch.stack(((x >> even) & 0xFFFF, (x >> odd) & 0xFFFF), 1).reshape(-1)[:n]).float() + 0.5) / 65536.0  # noqa: E731
    return both(0, 32), both(16, 40)


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 32)


def _decode(code, scale):
    n = code.numel()
    s = (scale.int() << 23).view(torch.float32)  # scale byte 0: a block of zeros
    return (_blocks(code).view(torch.float8_e4m3fn).float() * s[:, None]).view(-1)[:n]


def _encode(x, u, positive):
    n = x.numel()
    b, u = _blocks(x), _blocks(u)
    fine = torch.isfinite(b)
    a = torch.where(fine, b.abs(), 0.0)
    f, e = torch.frexp(a.amax(1))
    byte = torch.where(f > 0, torch.clamp(e - torch.where(f <= 0.875, 9, 8) + 127, 1, 254), 0)
    y = torch.ldexp(a, 127 - byte[:, None])
    step = torch.exp2((torch.clamp(torch.frexp(y)[1] - 1, min=-6) - 3).float())
    r = torch.floor(y / step + u) * step
    if positive:
        r = torch.where(a > 0, r.clamp_min(2.0 ** -9), r)
    r = torch.where(fine, torch.copysign(r, b), math.nan)
    return r.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:n], byte.to(torch.uint8)


def _adamw_plain(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    (b1, b2), t, lr = h["betas"], h["step"], h["lr"]
    for j, ((o, n), (bo, bn)) in enumerate(zip(s["spans"], s["bspans"])):
        p, at, sc = s["param"][o:o + n], slice(o, o + n), slice(bo, bo + bn)
        g = s["grad"][at].float() * h["grad_scale"]
        m = _decode(s["m"][at], s["m_scale"][sc]) if eight else s["m"][at]
        r = _decode(s["v"][at], s["v_scale"][sc]) if eight else None
        v = r * r if eight else s["v"][at]
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * (1.0 - b2) * g
        r = torch.sqrt(v)
        new = p.float() * (1.0 - lr * h["weight_decay"]) - lr / (1.0 - b1 ** t) * (m / (r * (1.0 / math.sqrt(1.0 - b2 ** t)) + h["eps"]))
        s["param"][at] = new.to(p.dtype)
        if s["copy"] is not None:
            s["copy"][at] = new.to(torch.bfloat16)
        if eight:
            um, ur = _uniforms(h["seed"], t, j, n, p.device)
            s["m"][at], s["m_scale"][sc] = _encode(m, um, False)
            s["v"][at], s["v_scale"][sc] = _encode(r, ur, True)
        else:
            s["m"][at], s["v"][at] = m, v
    return _adamw_outputs(s)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    size = {"fp32": 4, "bf16": 2}
    if op == "route":
        n, pairs = case["T"] * case["E"], case["T"] * case["K"]
        return {"bytes": n * size[case["dtype"]] + 16 * pairs + 4 * case["E"] * (2 if case["bias"] else 1), "flops": 4 * n + 4 * pairs}
    if op == "route_backward":
        n, pairs = case["T"] * case["E"], case["T"] * case["K"]
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": (n * (2 if dense else 1) + (0 if dense else pairs)) * size[case["dtype"]] + 8 * pairs, "flops": (6 * n if dense else 0) + 8 * pairs}
    if op in ("combine", "combine_backward"):
        T, K, H = case["T"], case["K"], case["H"]
        rows = T * K - _dropped(case)
        bytes_ = T * H * size[case["out"]] + 4 * T * K * (2 if case["weights"] else 1)
        if op == "combine":
            return {"bytes": bytes_ + rows * H * size[case["y"]], "flops": 2 * rows * H}
        more = rows * H * size[case["y"]] + 4 * T * K if case["weights"] else 0
        return {"bytes": bytes_ + more + rows * H * size[case["out"]], "flops": (3 if case["weights"] else 0) * rows * H}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 4 / 32
    return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + state + (2 if case["copy"] else 0)), "flops": 16 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _route_exact, "route_backward": _route_backward_exact, "combine": _combine_exact,
            "combine_backward": _combine_backward_exact, "adamw": _adamw_exact}[case["op"]](s)


def _route_exact(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["n_group"]
    l = s["logits"].float().cpu().numpy().astype(np.float64)
    off = l <= LOWEST
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            p = np.where(l >= 0, 1 / (1 + np.exp(-l)), np.exp(l) / (1 + np.exp(l)))
        else:
            top = np.where(off, -np.inf, l).max(1, keepdims=True)
            p = np.exp(l - np.where(np.isfinite(top), top, 0))
            p[off] = 0
            p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    p[off] = 0
    rank = p if s["bias"] is None else p + s["bias"].cpu().numpy().astype(np.float64)
    allowed = ~off
    if G > 1:
        per = np.where(off, -np.inf, rank).reshape(T, G, E // G)
        first = per.max(2)
        total = first.copy()
        if c["group_top"] == 2 and E // G > 1:
            second = np.partition(per, E // G - 2, axis=2)[:, :, E // G - 2]
            total = total + np.where(np.isfinite(second), second, 0)
        lead = np.argsort(-total, axis=1, kind="stable")[:, : c["topk_group"]]
        use = np.zeros((T, G), bool)
        np.put_along_axis(use, lead, True, 1)
        allowed &= np.repeat(use, E // G, axis=1)
    order = np.argsort(np.where(allowed, -(l if s["bias"] is None else rank), np.inf), axis=1, kind="stable")[:, :K]
    ok = np.take_along_axis(allowed, order, 1)
    w = np.where(ok, np.take_along_axis(p, order, 1), 0)
    if c["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    w = w * c["scale"]
    idx = np.where(ok, order, -1)
    pairs = np.flatnonzero(idx.reshape(-1) >= 0)
    of = idx.reshape(-1)[pairs]
    place = pairs[np.lexsort((pairs, of))]
    slot, token = np.full(T * K, -1), np.full(T * K, -1)
    slot[place] = np.arange(len(place))
    token[: len(place)] = place // K
    i32 = np.int32
    return {"idx": idx.astype(i32), "weights": w, "group_end": np.cumsum(np.bincount(of, minlength=E)).astype(i32),
            "row_token": token.astype(i32), "slot": slot.reshape(T, K).astype(i32)}


def _route_backward_exact(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_()
    off = x.detach() <= LOWEST
    there = s["idx"] >= 0
    i = s["idx"].long().clamp_min(0)
    if c["score"] == "sigmoid":
        score = torch.sigmoid(torch.where(off, -1e9, x))
    else:
        score = torch.softmax(torch.where(off, -1e9, x), 1)
    w = torch.where(there, score.gather(1, i), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    (w * c["scale"] * torch.where(there, s["dweights"].double(), 0.0)).sum().backward()
    return torch.where(off, 0.0, x.grad)


def _combine_exact(s):
    T, K = s["slot"].shape
    out = torch.zeros(T, s["y"].shape[1], dtype=torch.float64, device=DEV)
    for k in range(K):
        at = torch.nonzero(s["slot"][:, k] >= 0)[:, 0]
        w = 1.0 if s["weights"] is None else s["weights"][at, k].double()[:, None]
        out[at] += w * s["y"][s["slot"][at, k].long()].double()
    return out


def _combine_backward_exact(s):
    T, K = s["slot"].shape
    d = s["dout"].double()
    dy = torch.zeros(s["rows"], d.shape[1], dtype=torch.float64, device=DEV)
    dw = None if s["weights"] is None else torch.zeros(T, K, dtype=torch.float64, device=DEV)
    for k in range(K):
        at = torch.nonzero(s["slot"][:, k] >= 0)[:, 0]
        row = s["slot"][at, k].long()
        dy[row] = d[at] * (1.0 if s["weights"] is None else s["weights"][at, k].double()[:, None])
        if dw is not None:
            dw[at, k] = (s["y"][row].double() * d[at]).sum(1)
    return {"dy": dy, "dweights": dw}


def _adamw_exact(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    (b1, b2), t = h["betas"], h["step"]
    f64 = torch.float64
    out = {"param": s["param"].to(f64), "m": s["m"].to(f64), "v": s["v"].to(f64)}
    if s["copy"] is not None:
        out["copy"] = s["copy"].to(f64)
    if eight:
        out["m_scale"] = s["m_scale"].view(torch.float8_e8m0fnu).to(f64)
        out["v_scale"] = s["v_scale"].view(torch.float8_e8m0fnu).to(f64)
        pos = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).to(f64)  # the magnitudes, ascending
    chunk = 1 << 25
    for j, ((o, n), (bo, _)) in enumerate(zip(s["spans"], s["bspans"])):
        key = (h["seed"] + 0x9E3779B9 * t + 0xBB67AE85 * (j + 1)) % 2 ** 32
        for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
            key = ((key ^ (key >> shift)) * factor) % 2 ** 32
        key ^= key >> 16
        for c0 in range(0, n, chunk):
            k = min(chunk, n - c0)
            at, nb = slice(o + c0, o + c0 + k), -(-k // 32)
            blk = slice(bo + c0 // 32, bo + c0 // 32 + nb)
            g = s["grad"][at].to(f64) * h["grad_scale"]
            m, r = s["m"][at], s["v"][at]
            if eight:
                of = torch.arange(k, device=DEV) // 32
                m = m.view(torch.float8_e4m3fn).to(f64) * torch.exp2(s["m_scale"][blk].to(f64) - 127)[of]
                v = (r.view(torch.float8_e4m3fn).to(f64) * torch.exp2(s["v_scale"][blk].to(f64) - 127)[of]) ** 2
            else:
                m, v = m.to(f64), r.to(f64)
            m = b1 * m + (1 - b1) * g
            v = b2 * v + (1 - b2) * g ** 2
            p = s["param"][at].to(f64) * (1 - h["lr"] * h["weight_decay"])
            p = p - h["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + h["eps"])
            out["param"][at] = p
            if s["copy"] is not None:
                out["copy"][at] = p
            if not eight:
                out["m"][at], out["v"][at] = m, v
                continue
            i = torch.arange(c0, c0 + k, device=DEV)
            z = (key + (i // 2) * 0x9E3779B9 + (i // 2 // 2 ** 32) * 0x243F6A89) & MASK32
            z = ((z ^ (z >> 15)) * 0x6A09E667) & MASK32
            z = (z ^ (z >> 13)) * 0xBB67AE85
            for name, x, even, odd in (("m", m, 0, 32), ("v", v.sqrt(), 16, 40)):
                u = (((z >> torch.where(i % 2 == 0, even, odd)) & 0xFFFF).to(f64) + 0.5) / 65536
                a = x.abs()
                top = torch.cat((a, a.new_zeros(nb * 32 - k))).view(nb, 32).amax(1)
                e = torch.where(top > 0, torch.clamp(torch.ceil(torch.log2(top / 448)), -126, 127), -127.0)
                y = a / torch.exp2(e)[of]
                lo = torch.searchsorted(pos, y, right=True) - 1
                hi = (lo + 1).clamp_max(126)
                gap = torch.where(hi > lo, pos[hi] - pos[lo], 1.0)
                code = torch.where((y - pos[lo]) / gap + u >= 1, hi, lo)
                if name == "v":
                    code = torch.where(a > 0, code.clamp_min(1), code)
                out[name][at] = torch.copysign(pos[code], x)
                out[name + "_scale"][blk] = torch.exp2(e)
    return out
