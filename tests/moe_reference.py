"""Plain 64-bit implementations of the router, expert order, combine and AdamW entry points (numpy, one row or element at
a time where that is clearest), for the tests; written from the definitions in include/mxq.h."""
import numpy as np

U32 = 2.0 ** -24    # half a step of fp32, relative
UBF16 = 2.0 ** -8   # of bf16
LOWEST = -3.3895313892515355e38


def route(logits, K, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalise=True, scale=1.0):
    """logits fp64 [T][E] -> idx int32, weights fp64 [T][K]."""
    T, E = logits.shape
    idx, weights = np.full((T, K), -1, np.int32), np.zeros((T, K))
    with np.errstate(all="ignore"):
        for t in range(T):
            l = logits[t]
            off = l <= LOWEST
            if score == "sigmoid":
                e = np.exp(-np.abs(l))
                s = np.where(l >= 0, 1.0, e) / (1.0 + e)
            else:
                e = np.where(off, 0.0, np.exp(l - np.max(l[~off], initial=-np.inf)))
                s = e / e.sum()
            s = np.where(off, 0.0, s)
            key = s if bias is None else s + bias
            key = np.where(np.isnan(key), -1e300, key)
            per = E // n_group
            groups = []
            for g in range(n_group):
                k = key[g * per:(g + 1) * per][~off[g * per:(g + 1) * per]]
                k = np.sort(k[k > -np.inf])[::-1][:group_top]
                groups.append(k.sum() if len(k) else -np.inf)
            kept = [g for g in sorted(range(n_group), key=lambda g: (-groups[g], g))[:topk_group]]
            order = l if bias is None else key
            order = np.where(np.isnan(order), -1e300, order)
            allowed = [e for e in range(E) if not off[e] and order[e] > -np.inf and e // per in kept and groups[e // per] > -np.inf]
            chosen = sorted(allowed, key=lambda e: (-order[e], e))[:K]
            w = s[chosen]
            if renormalise:
                w = w / w.sum() if w.sum() != 0 else np.zeros(len(w))
            idx[t, :len(chosen)], weights[t, :len(chosen)] = chosen, w * scale
    return idx, weights


def route_rows(logits, K, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalise=True, scale=1.0):
    """route of many rows at once; logits and keys finite or masked."""
    T, E = logits.shape
    off = logits <= LOWEST
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(logits))
            s = np.where(logits >= 0, 1.0, e) / (1.0 + e)
        else:
            e = np.where(off, 0.0, np.exp(logits - np.where(off, -np.inf, logits).max(1, keepdims=True)))
            s = e / e.sum(1, keepdims=True)
        s = np.where(off, 0.0, s)
        key = np.where(off, -np.inf, s if bias is None else s + bias)
        order = np.where(off, -np.inf, logits) if bias is None else key
        if n_group > 1:
            best = np.sort(key.reshape(T, n_group, -1), axis=2)[:, :, ::-1][:, :, :group_top]
            total = np.where(best[:, :, 0] > -np.inf, np.where(best > -np.inf, best, 0.0).sum(2), -np.inf)
            rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
            order = np.where((rank < topk_group).repeat(E // n_group, axis=1), order, -np.inf)
        chosen = np.argsort(-order, axis=1, kind="stable")[:, :K]
        there = np.take_along_axis(order, chosen, 1) > -np.inf
        w = np.where(there, np.take_along_axis(s, chosen, 1), 0.0)
        if renormalise:
            w = np.where(there, w / np.where(w.sum(1, keepdims=True) != 0, w.sum(1, keepdims=True), 1.0), 0.0)
    return np.where(there, chosen, -1).astype(np.int32), w * scale


def expert_order(idx, E):
    T, K = idx.shape
    flat = idx.reshape(-1)
    pairs = [i for e in range(E) for i in np.flatnonzero(flat == e)]
    slot, token = np.full(T * K, -1, np.int32), np.full(T * K, -1, np.int32)
    slot[pairs] = np.arange(len(pairs))
    token[:len(pairs)] = np.asarray(pairs, np.int64) // K
    ends = np.cumsum([(flat == e).sum() for e in range(E)]).astype(np.int32)
    return ends, token, slot.reshape(T, K)


def route_backward(logits, idx, dweights, score="softmax", renormalise=True, scale=1.0):
    """Gradient by the product and quotient rules: d w_k / d s_j, then d s_j / d l_e, with full matrices."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l, off = logits[t], logits[t] <= LOWEST
        ks = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E and not off[idx[t, k]]]
        if not ks:
            continue
        sel, g = idx[t, ks], dweights[t, ks] * scale
        if score == "softmax" and renormalise:  # the softmax of the chosen logits alone; the others cancel
            e = np.exp(l[sel] - l[sel].max())
            p = e / e.sum()
            out[t, sel] = g @ (np.diag(p) - np.outer(p, p))
            continue
        if score == "sigmoid":
            s = np.where(off, 0.0, 1.0 / (1.0 + np.exp(-np.where(off, 0.0, l))))
            ds_dl = np.diag(s * (1 - s))
        else:
            e = np.where(off, 0.0, np.exp(np.where(off, 0.0, l) - l[~off].max()))
            s = e / e.sum()
            ds_dl = np.diag(s) - np.outer(s, s)
        if renormalise:
            total = s[sel].sum()
            dw_ds = np.eye(len(sel)) / total - np.outer(s[sel], np.ones(len(sel))) / total ** 2
        else:
            dw_ds = np.eye(len(sel))
        out[t] = (g @ dw_ds) @ ds_dl[sel]
    return out


def route_backward_rows(logits, idx, dweights, score="softmax", renormalise=True, scale=1.0):
    """route_backward of many rows at once, by the closed forms."""
    T, E = logits.shape
    off = logits <= LOWEST
    there = (idx >= 0) & (idx < E)
    at = np.where(there, idx, 0)
    there &= ~np.take_along_axis(off, at, 1)
    g = np.where(there, dweights * scale, 0.0)
    out = np.zeros((T, E + 1))
    put = np.where(there, at, E)  # no gradient: the column past the last
    l = np.where(off, -np.inf, logits)
    x = np.where(there, np.take_along_axis(l, at, 1), -np.inf)
    sig = 1.0 / (1.0 + np.exp(-np.where(there, x, 0.0)))
    if score == "sigmoid" and not renormalise:
        np.put_along_axis(out, put, g * sig * (1.0 - sig), 1)
    elif renormalise:
        some = there.any(1, keepdims=True)
        p = np.where(there, sig if score == "sigmoid" else np.exp(x - np.where(some, x.max(1, keepdims=True), 0.0)), 0.0)
        p = p / np.where(some, p.sum(1, keepdims=True), 1.0)
        d = p * (g - (p * g).sum(1, keepdims=True))
        np.put_along_axis(out, put, d * (1.0 - sig) if score == "sigmoid" else d, 1)
    else:
        top = l.max(1, keepdims=True)
        e = np.where(off, 0.0, np.exp(l - np.where(top > -np.inf, top, 0.0)))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
        np.put_along_axis(out, put, g, 1)
        out[:, :E] = s * (out[:, :E] - (s * out[:, :E]).sum(1, keepdims=True))
    return out[:, :E]


def mix(x):
    x = (x ^ (x >> 16)) * 0x6A09E667 % 2 ** 32
    x = (x ^ (x >> 15)) * 0xBB67AE85 % 2 ** 32
    return x ^ (x >> 16)


def uniforms(seed, step, tensor, n, first=0):
    """(u for m, u for r) of elements first .. first + n - 1 (first even)."""
    key = mix((seed + 0x9E3779B9 * step + 0xBB67AE85 * (tensor + 1)) % 2 ** 32)
    q = np.arange(first // 2, (first + n + 1) // 2, dtype=np.uint64)
    m32 = np.uint64(0xFFFFFFFF)
    x = (np.uint64(key) + (q & m32) * np.uint64(0x9E3779B9) + (q >> np.uint64(32)) * np.uint64(0x243F6A89)) & m32
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667)) & m32
    p = (x ^ (x >> np.uint64(13))) * np.uint64(0xBB67AE85)
    f = lambda a, b: (np.stack([(p >> np.uint64(s)) & np.uint64(0xFFFF) for s in (a, b)], 1).reshape(-1)[:n] + 0.5) / 65536  # noqa: E731
    return f(0, 32), f(16, 40)


E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def decode(codes, scales):
    v = np.append(E4M3, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return v * np.where(scales == 0, 0.0, 2.0 ** (scales.astype(np.float64) - 127)).repeat(32)[:len(codes)]


def encode(x, u, positive=False):
    """(codes, scales, unsure, scale_unsure): unsure marks elements whose rounding 2^-16 of a step decides, and blocks
    whose largest magnitude is within 2^-20 of a scale's border."""
    n = len(x)
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0)
    top = np.pad(a, (0, -n % 32)).reshape(-1, 32).max(1)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(top / 448.0))
    near = np.abs(top / 448.0 / 2.0 ** np.round(np.where(top > 0, np.log2(np.maximum(top, 1e-300) / 448.0), 0)) - 1) < 2.0 ** -20
    scales = np.where(top > 0, np.clip(e + 127, 1, 254), 0).astype(np.uint8)
    y = a / (2.0 ** (np.maximum(scales, 1).astype(np.float64) - 127)).repeat(32)[:n]
    lo = np.clip(np.searchsorted(E4M3, y, side="right") - 1, 0, 126)
    gap = np.where(lo < 126, E4M3[np.minimum(lo + 1, 126)] - E4M3[lo], 1.0)
    f = (y - E4M3[lo]) / gap
    code = np.where(f + u >= 1, lo + 1, lo)
    if positive:
        code = np.where((a > 0) & (code == 0), 1, code)
    code = np.where(fine, code, 127) | np.where(np.signbit(x) & fine, 128, 0)
    return code.astype(np.uint8), scales, np.abs(f + u - 1) < 2.0 ** -16, near


def adamw(p, g, m, v, lr, betas, eps, weight_decay, step, grad_scale):
    """fp64 (p, m, v) after the step, and the error bounds of an fp32 evaluation (each operation and each constant
    rounded once)."""
    b1, b2 = betas
    g = g * grad_scale
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    dm = 4 * U32 * (np.abs(b1 * m) + np.abs((1 - b1) * g)) + 2.0 ** -148
    dv = 6 * U32 * v1 + 2.0 ** -147
    den = np.sqrt(v1) / np.sqrt(1 - b2 ** step) + eps
    alpha = lr / (1 - b1 ** step)
    p1 = p * (1 - lr * weight_decay) - alpha * m1 / den
    # r: half of v's error and one ulp; the scaling, the sum, the quotient (one ulp) and the product: 2 u each at most
    dr = np.sqrt(v1 + dv) - np.sqrt(np.maximum(v1 - dv, 0)) + 2 * U32 * np.sqrt(v1)
    dden = dr / np.sqrt(1 - b2 ** step) + 4 * U32 * den
    dp = alpha * (dm / den + np.abs(m1) * dden / den ** 2 + 8 * U32 * np.abs(m1) / den) + U32 * (3 * np.abs(p) + 2 * np.abs(p1))
    return p1, m1, v1, dp, dm, dv
