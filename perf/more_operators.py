"""Cases of FP8 with one fp32 scale for every block of 128 (the quantisers, the dense and the grouped products that take
their operands) and of the Muon step of weight matrices (momentum and Newton-Schulz orthogonalisation).

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through the
library's entry points, on the inputs that ``prepare`` makes; ``exact`` gives the same outputs from the operators'
definitions in 64 bits; ``work`` gives the bytes and operations a pass cannot do without.

Definitions
  quantise  the matrix in blocks of 1 x 128 (128 along the reduction axis) or 128 x 128, the last ones short:
            amax = max(largest |x| of the block, 2^-100), scale = amax / 448, code = e4m3(x * 448 / amax), to nearest even.
            "row" copy: codes [R][ceil128(C)], scales [C / 128][R] (1 x 128) or [C / 128][R / 128]; "colT" copy: the same
            of the transpose.  Grouped: blocks run down the rows of each group and restart with it, so group g has
            ceil128(m_g) columns of the colT copy.  Codes past a row's (or a group's) end are 0.
  gemm      C[m][n] = sum over blocks b of 128: sA[b][m] sB[b][n] sum over k in b of A[m][k] B[n][k].
            ragged M: row m of group g takes B[g]; ragged K: C[g] is the sum over group g's blocks.
  muon      m' = beta m + (1 - beta) g; u = (1 - beta) g + beta m' (Nesterov) or m';
            X = u / (|u|_F + eps); five times X = a X + (b A + c A^2) X with A = X X^T; p' = p (1 - lr wd) - lr scale X.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
BLOCK = 128
FLOOR = 2.0 ** -100  # smallest amax a block's scale is taken from
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step's activations before a product; latency counts
        {"name": "quantize_decode", "op": "quantize", "batch": 1, "R": 7, "C": 7168, "tile": 1, "row": True, "colT": False,
         "groups": 0, "dtype": "bf16"},
        # the experts' output gradients in expert order: rows for the input gradient, tokens for the weight gradient
        {"name": "quantize_grouped_train", "op": "quantize", "batch": 1, "R": 131072, "C": 4096, "tile": 1, "row": True,
         "colT": True, "groups": 32, "dtype": "bf16"},
        # the weights of the 32 local experts, for the forward and for the input gradient
        {"name": "quantize_experts", "op": "quantize", "batch": 32, "R": 7168, "C": 4096, "tile": 128, "row": True, "colT": True,
         "groups": 0, "dtype": "bf16"},
        # one decoding step through a linear layer: the weight is read once for a few rows
        {"name": "gemm_decode", "op": "gemm", "M": 7, "K": 7168, "N": 4096, "tile": 128, "out": "bf16"},
        # the dense linear layer's forward
        {"name": "gemm_train", "op": "gemm", "M": 8192, "K": 7168, "N": 18432, "tile": 128, "out": "bf16"},
        # a decoding step of 8 tokens, top 8, through the 32 local experts
        {"name": "grouped_decode", "op": "ragged_m", "T": 64, "K": 7168, "N": 4096, "groups": 32, "out": "bf16"},
        # the MoE layer's routed rows through the 32 local experts
        {"name": "grouped_train", "op": "ragged_m", "T": 131072, "K": 7168, "N": 4096, "groups": 32, "out": "bf16"},
        # the experts' weight gradients in fp32, as the optimiser takes them
        {"name": "wgrad_train", "op": "ragged_k", "T": 131072, "M": 7168, "N": 4096, "groups": 32, "out": "fp32"},
        # a small layer of odd sizes with few tokens an expert, bf16 gradients
        {"name": "wgrad_odd", "op": "ragged_k", "T": 4099, "M": 511, "N": 1237, "groups": 16, "out": "bf16"},
        # the expert weights of a small MoE layer, fp32 with the bf16 copy that the quantiser reads
        {"name": "muon_small", "op": "muon", "batch": 32, "R": 512, "C": 256, "param": "fp32", "grad": "fp32", "nesterov": True,
         "copy": True},
        # four experts' weights (one of eight ranks that share 32), the weight-gradient product's fp32 output
        {"name": "muon_experts", "op": "muon", "batch": 4, "R": 7168, "C": 4096, "param": "fp32", "grad": "fp32",
         "nesterov": True, "copy": True},
        # the same with weights and gradients held in bf16
        {"name": "muon_experts_bf16", "op": "muon", "batch": 4, "R": 7168, "C": 4096, "param": "bf16", "grad": "bf16",
         "nesterov": True, "copy": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["quantize", "quantize", "gemm", "gemm", "ragged_m", "ragged_m", "ragged_k", "muon", "muon"])
    coin = lambda p=0.5: rng.random() < p  # noqa: E731
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "quantize":
        axes = rng.choice([(True, False), (False, True), (True, True)])
        c = {"op": op, "R": _log(rng, 1, 32768), "C": _log(rng, 64, 7168), "row": axes[0], "colT": axes[1], "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        kind = rng.choice(["rows", "tiles", "grouped"])
        return c | {"tile": 128 if kind == "tiles" else 1, "batch": rng.randint(1, 8) if kind == "tiles" else 1,
                    "groups": _log(rng, 1, 64) if kind == "grouped" else 0}
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 64, 7168), "N": _log(rng, 64, 8192), "tile": rng.choice([1, 128, 128]), "out": out}
    if op == "ragged_m":
        return {"op": op, "T": _log(rng, 1, 32768), "K": _log(rng, 64, 4096), "N": _log(rng, 64, 4096), "groups": _log(rng, 1, 64), "out": out}
    if op == "ragged_k":
        return {"op": op, "T": _log(rng, 1, 32768), "M": _log(rng, 64, 4096), "N": _log(rng, 64, 4096), "groups": _log(rng, 1, 32), "out": out}
    param = rng.choice(["fp32", "bf16"])
    return {"op": op, "batch": _log(rng, 1, 16), "R": _log(rng, 16, 2048), "C": _log(rng, 16, 2048), "param": param,
            "grad": rng.choice(["fp32", "bf16"]), "nesterov": coin(), "copy": param == "fp32" and coin()}


# ------------------------------------------------------------------ inputs
def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _up(n):
    return -(-n // BLOCK) * BLOCK


def _sizes(T, groups, seed):
    """Rows of each group: popularity falling as 1 / (e + 1)^1.1 in a shuffled order, so some groups may get none."""
    r = np.random.default_rng(seed)
    p = r.permutation((np.arange(groups) + 1.0) ** -1.1)
    return r.multinomial(T, p / p.sum()).tolist()


def _ends(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device=DEV)


def _activations(rows, cols, g, dtype):
    """N(0, 1) with a few columns that are 20 times as large."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x[:, torch.randint(0, cols, (max(1, cols // 512),), generator=g, device=DEV)] *= 20.0
    return x.to(dtype)


def _operand(x, tile):
    """Codes (uint8) and scales of the row copy, as a program holds them after quantising."""
    q, s = _quantize_plain(x, tile)
    return q.view(torch.uint8), s


def _gradient(case, g, dtype):
    """A gradient: a few strong directions over noise."""
    B, R, C = case["batch"], case["R"], case["C"]
    k = max(1, min(R, C) // 32)
    u, v = torch.randn(B, R, k, generator=g, device=DEV), torch.randn(B, k, C, generator=g, device=DEV)
    return (torch.bmm(u, v).mul_(k ** -0.5) + torch.randn(B, R, C, generator=g, device=DEV)).mul_(1e-3).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        B, R, C = case["batch"], case["R"], case["C"]
        if case["tile"] == 128:
            s["x"] = torch.randn(B, R, C, generator=g, device=DEV).mul_(0.02).to(_dt(case["dtype"]))
        else:
            s["x"] = _activations(R, C, g, _dt(case["dtype"]))
        if case["groups"]:
            s["sizes"] = _sizes(R, case["groups"], seed)
            s["group_end"] = _ends(s["sizes"])
            s["ldq"] = max(BLOCK, sum(_up(m) for m in s["sizes"]))
        s["out"] = _quantize_buffers(case, s)
        return s
    if op == "gemm":
        s["A"], s["sA"] = _operand(_activations(case["M"], case["K"], g, torch.bfloat16), 1)
        s["B"], s["sB"] = _operand(torch.randn(case["N"], case["K"], generator=g, device=DEV).mul_(0.02), case["tile"])
        return s
    if op == "ragged_m":
        G, N, K = case["groups"], case["N"], case["K"]
        s["sizes"] = _sizes(case["T"], G, seed)
        s["group_end"] = _ends(s["sizes"])
        s["A"], s["sA"] = _operand(_activations(case["T"], K, g, torch.bfloat16), 1)
        pairs = [_operand(torch.randn(N, K, generator=g, device=DEV).mul_(0.02), 128) for _ in range(G)]
        s["B"], s["sB"] = torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])
        return s
    if op == "ragged_k":
        s["sizes"] = _sizes(case["T"], case["groups"], seed)
        s["group_end"] = _ends(s["sizes"])
        for name, cols in (("A", case["M"]), ("B", case["N"])):
            x = _spread(_activations(case["T"], cols, g, torch.bfloat16), s["sizes"])
            s[name], s["s" + name] = _operand(x.t().contiguous(), 1)
            del x
        return s
    s["param"] = torch.randn(case["batch"], case["R"], case["C"], generator=g, device=DEV).mul_(0.02).to(_dt(case["param"]))
    s["grad"] = _gradient(case, g, _dt(case["grad"]))
    s["m"] = _gradient(case, g, torch.float32)
    s["copy"] = torch.zeros_like(s["param"], dtype=torch.bfloat16) if case["copy"] else None
    s["hyper"] = {"lr": 1e-3, "momentum": 0.95, "weight_decay": 0.1, "scale": 0.2 * math.sqrt(max(case["R"], case["C"]))}
    return s


def _quantize_buffers(case, s):
    """The copies that a program has allocated: rows, and columns of the transpose."""
    B, R, C, tile = case["batch"], case["R"], case["C"], case["tile"]
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)  # noqa: E731
    f32 = lambda *shape: torch.zeros(shape, device=DEV)  # noqa: E731
    lead = (B,) if tile == 128 else ()
    Rp = s["ldq"] if case["groups"] else _up(R)
    out = {}
    if case["row"]:
        out["q_row"], out["s_row"] = u8(*lead, R, _up(C)), f32(*lead, _up(C) // BLOCK, -(-R // tile))
    if case["colT"]:
        out["q_colT"], out["s_colT"] = u8(*lead, C, Rp), f32(*lead, Rp // BLOCK, -(-C // tile))
    return out


def _spread(x, sizes):
    """Rows of x with each group padded to a multiple of 128 with zeros."""
    P = max(BLOCK, sum(_up(m) for m in sizes))
    at = np.concatenate([np.arange(m) + o for m, o in zip(sizes, np.cumsum([0] + [_up(m) for m in sizes[:-1]]))]).astype(np.int64)
    y = torch.zeros(P, x.shape[1], dtype=x.dtype, device=x.device)
    y[torch.from_numpy(at).to(x.device)] = x
    return y


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _codes(out):
    """The copies, 8-bit codes as the values they stand for."""
    return {k: v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v for k, v in out.items() if isinstance(v, torch.Tensor)}


def _run_own(s):
    from moe_grouped_gemm_mxq_amd import mxq

    c = s["case"]
    if c["op"] == "quantize":
        axes = (mxq.MXQ_AXIS_ROW if c["row"] else 0) | (mxq.MXQ_AXIS_COLT if c["colT"] else 0)
        if c["groups"]:
            return _codes(mxq.quantize128_grouped(s["x"], s["group_end"], axes, ldq=s["ldq"], out=s["out"]))
        return _codes(mxq.quantize128(s["x"], axes, tile=c["tile"], out=s["out"]))
    if c["op"] == "gemm":
        return mxq.gemm128(s["A"], s["sA"], s["B"], s["sB"], dtype=_dt(c["out"]))
    if c["op"] in ("ragged_m", "ragged_k"):
        mode = mxq.MXQ_GG_RAGGED_M if c["op"] == "ragged_m" else mxq.MXQ_GG_RAGGED_K
        return mxq.grouped_gemm128(mode, s["A"], s["sA"], s["B"], s["sB"], s["group_end"], dtype=_dt(c["out"]))
    if "plan" not in s:  # a program makes it once, with its tensors
        s["plan"] = mxq.Muon([s["param"]], [s["grad"]], [s["m"]], copies=[s["copy"]])
    s["plan"].step(nesterov=c["nesterov"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS, **s["hyper"])
    return _muon_outputs(s)


def _muon_outputs(s):
    out = {"param": s["param"], "m": s["m"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


def _run_plain(s):
    return {"quantize": _quantize_case, "gemm": _gemm_plain, "ragged_m": _ragged_m_plain, "ragged_k": _ragged_k_plain,
            "muon": _muon_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------ plain forms
def _quantize_plain(x, tile):
    """Codes (float8) [.., R][ceil128(C)] and scales [.., C / 128][R / tile] of the row copy of x [.., R][C]."""
    R, C = x.shape[-2:]
    v = torch.nn.functional.pad(x.float(), (0, -C % BLOCK, 0, -R % tile))
    v = v.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, tile))  # [.., R / tile, tile, C / 128, 128]
    amax = v.abs().amax((-3, -1), keepdim=True).clamp_min(FLOOR)
    # (x * 7/8 is exact in 32 bits for a bf16 x, so a quotient half way between two codes comes out as it is)
    q = (v * 0.875 / (amax / 512.0)).to(torch.float8_e4m3fn).flatten(-2).flatten(-3, -2)[..., :R, :]
    return q.contiguous(), (amax / 448.0)[..., 0, :, 0].mT.contiguous()


def _quantize_case(s):
    c, x, out = s["case"], s["x"], {}
    if c["row"]:
        out["q_row"], out["s_row"] = _quantize_plain(x, c["tile"])
    if c["colT"]:
        t = _spread(x, s["sizes"]) if c["groups"] else x
        out["q_colT"], out["s_colT"] = _quantize_plain(t.mT, c["tile"])
    return out


def _values(q, s):
    """fp32 values [rows][K] of codes and scales [K / 128][rows] or [K / 128][rows / 128]."""
    rows = q.shape[0]
    scale = s.t() if s.shape[1] == rows else s.t().repeat_interleave(BLOCK, 0)[:rows]
    return (q.view(torch.float8_e4m3fn).float().unflatten(1, (-1, BLOCK)) * scale[:, :, None]).flatten(1)


def _gemm_plain(s):
    return (_values(s["A"], s["sA"]) @ _values(s["B"], s["sB"]).t()).to(_dt(s["case"]["out"]))


def _ragged_m_plain(s):
    a = _values(s["A"], s["sA"]).split(s["sizes"])
    y = [x @ _values(q, t).t() for x, q, t in zip(a, s["B"], s["sB"])]
    return torch.cat(y).to(_dt(s["case"]["out"]))


def _ragged_k_plain(s):
    a, b = _values(s["A"], s["sA"]), _values(s["B"], s["sB"])
    spans = [_up(m) for m in s["sizes"]]
    rest = a.shape[1] - sum(spans)  # (no rows at all: one block of zeros)
    y = [x @ z.t() for x, z in zip(a.split(spans + [rest], 1)[:-1], b.split(spans + [rest], 1))]
    return torch.stack(y).to(_dt(s["case"]["out"]))


def _muon_plain(s):
    c, h = s["case"], s["hyper"]
    beta = h["momentum"]
    g = s["grad"].float()
    s["m"].mul_(beta).add_(g, alpha=1 - beta)
    u = (1 - beta) * g + beta * s["m"] if c["nesterov"] else s["m"].clone()
    wide = c["R"] <= c["C"]
    x = u if wide else u.mT.contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = torch.bmm(x, x.mT.contiguous())
        B = COEFFICIENTS[1] * A + COEFFICIENTS[2] * torch.bmm(A, A)
        x = COEFFICIENTS[0] * x + torch.bmm(B, x)
    p = s["param"].float() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * h["scale"] * (x if wide else x.mT)
    s["param"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    return _muon_outputs(s)


# ------------------------------------------------------------------ work of a pass
def work(case):
    op = case["op"]
    wide = lambda name: 4 if name == "fp32" else 2  # noqa: E731
    if op == "quantize":
        n = case["batch"] * case["R"] * case["C"]
        copies = case["row"] + case["colT"]
        return {"bytes": n * (wide(case["dtype"]) + copies * (1 + 4 / (BLOCK * case["tile"]))), "flops": 4 * n * copies}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * _up(K) + wide(case["out"]) * M * N, "flops": 2 * M * N * K}
    if op == "ragged_m":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": (T + min(case["groups"], T) * N) * _up(K) + wide(case["out"]) * T * N, "flops": 2 * T * N * K}
    if op == "ragged_k":
        T, M, N = case["T"], case["M"], case["N"]
        return {"bytes": (M + N) * T + wide(case["out"]) * case["groups"] * M * N, "flops": 2 * T * M * N}
    B, R, C = case["batch"], case["R"], case["C"]
    lo, hi = min(R, C), max(R, C)
    moved = 2 * wide(case["param"]) + wide(case["grad"]) + 2 * 4 + (2 if case["copy"] else 0)
    # of the symmetric products one half
    return {"bytes": B * R * C * moved, "flops": B * STEPS * (lo * lo * hi + lo * lo * lo + 2 * lo * lo * hi)}


# ------------------------------------------------------------------ exact, in 64 bits, from the definitions
def _e4m3_table():
    """Values of the 256 codes: sign, 4 exponent bits (bias 7), 3 of mantissa; the all-ones code is NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return torch.from_numpy(np.where(c & 128, -v, v)).to(DEV)


def _nearest_e4m3(y):
    """y rounded to the nearest value of E4M3, ties to even, in 64 bits: steps of 2^(exponent - 3), no smaller than 2^-9."""
    _, e = torch.frexp(y)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_copy(x, tile):
    """(values, scales) of the row copy of one matrix, whole rows of blocks at a time."""
    R, C = x.shape
    values = torch.zeros(R, _up(C), dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.zeros(_up(C) // BLOCK, -(-R // tile), dtype=torch.float64, device=x.device)
    for b in range(_up(C) // BLOCK):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].double()
        top = part.abs().amax(1)
        if tile > 1:
            top = torch.cat([top, top.new_zeros(-R % tile)]).view(-1, tile).amax(1)
        top = torch.clamp(top, min=FLOOR)
        scales[b] = top / 448.0
        each = top.repeat_interleave(tile)[:R, None]
        values[:, b * BLOCK:b * BLOCK + part.shape[1]] = _nearest_e4m3(part * 448.0 / each).to(torch.float8_e4m3fn)  # (holds them)
    return values, scales


def _exact_quantize(case, s):
    out = {}
    x = s["x"]
    for row, name in ((True, "row"), (False, "colT")):
        if not case[name]:
            continue
        if x.dim() == 3:
            got = [_exact_copy(m if row else m.t(), case["tile"]) for m in x]
            q, t = torch.stack([v[0].view(torch.uint8) for v in got]), torch.stack([v[1] for v in got])
        elif row or not case["groups"]:
            q, t = _exact_copy(x if row else x.t(), case["tile"])
            q = q.view(torch.uint8)
        else:  # each group by itself
            got = [_exact_copy(part.t(), 1) for part in x.split(s["sizes"]) if part.shape[0]]
            q, t = torch.cat([v[0].view(torch.uint8) for v in got], 1), torch.cat([v[1] for v in got])
        out["q_" + name], out["s_" + name] = q.view(torch.float8_e4m3fn), t
    return out


def _exact_values(q, s, table):
    """64-bit values of an operand, block by block."""
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    of = torch.arange(q.shape[0], device=q.device)
    of = of if s.shape[1] == q.shape[0] else of // BLOCK
    for b in range(q.shape[1] // BLOCK):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        out[:, cols] = table[q[:, cols].int()] * s[b].double()[of][:, None]
    return out


def _exact_products(case, s):
    table = _e4m3_table()
    if case["op"] == "gemm":
        return _exact_values(s["A"], s["sA"], table) @ _exact_values(s["B"], s["sB"], table).t()
    if case["op"] == "ragged_m":
        out = torch.empty(case["T"], case["N"], dtype=torch.float64, device=DEV)
        at = 0
        for g, m in enumerate(s["sizes"]):
            if m:
                a = _exact_values(s["A"][at:at + m], s["sA"][:, at:at + m], table)
                out[at:at + m] = a @ _exact_values(s["B"][g], s["sB"][g], table).t()
            at += m
        return out
    out = torch.zeros(case["groups"], case["M"], case["N"], dtype=torch.float64, device=DEV)
    at = 0
    for g, m in enumerate(s["sizes"]):
        if m:
            cols, blocks = slice(at, at + _up(m)), slice(at // BLOCK, (at + _up(m)) // BLOCK)
            a = _exact_values(s["A"][:, cols], s["sA"][blocks], table)
            out[g] = a @ _exact_values(s["B"][:, cols], s["sB"][blocks], table).t()
        at += _up(m)
    return out


def _exact_muon(case, s):
    h, a, b, c = s["hyper"], *COEFFICIENTS
    beta = h["momentum"]
    out = {"param": torch.empty(s["param"].shape, dtype=torch.float64, device=DEV), "m": torch.empty(s["m"].shape, dtype=torch.float64, device=DEV)}
    for i in range(case["batch"]):
        g = s["grad"][i].double()
        m = beta * s["m"][i].double() + (1 - beta) * g
        u = (1 - beta) * g + beta * m if case["nesterov"] else m
        x = u / (torch.linalg.vector_norm(u) + EPS)
        if case["R"] > case["C"]:  # the smaller products; the result is the same
            x = x.t().contiguous()
        for _ in range(STEPS):
            A = x @ x.t()
            x = a * x + (b * A + c * (A @ A)) @ x
        out["param"][i] = s["param"][i].double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * h["scale"] * (x.t() if case["R"] > case["C"] else x)
        out["m"][i] = m
    if case["copy"]:
        out["copy"] = out["param"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(case, s)
    if case["op"] == "muon":
        return _exact_muon(case, s)
    return _exact_products(case, s)
