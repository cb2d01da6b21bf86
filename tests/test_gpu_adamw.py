"""AdamW steps of many tensors against 64-bit references.  Bounds: moe_reference.adamw counts the half steps of an fp32
evaluation; MXFP8 codes have to be those of the reference except where 2^-16 of an E4M3 step decides the rounding.  They
round r from 64 bits (a sum of positive terms: off by less than 8 half steps, 2^-21, and an E4M3 step is at least 2^-4 of
the value) and m from the fp32 products and sum that the entry point documents, since 64 bits differ from those by more
where the two products cancel."""
import numpy as np
import pytest
import torch

import moe_reference as ref
from gpu_util import host, mxq

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1, step=7, grad_scale=0.25, seed=1234)
REF = {k: v for k, v in HYPER.items() if k != "seed"}
SIZES = [1, 2, 31, 32, 33, 64, 255, 1000, 4095, 4096, 4097, 20011]


def f64(t):
    return t.detach().cpu().double().numpy()


def tensors(sizes, pdt, gdt, bits, seed=0, offset=0):
    """Tensors cut out of longer ones at `offset` elements, so that alignments vary."""
    g = torch.Generator().manual_seed(seed)
    cut = lambda x: x.cuda()[offset:]  # noqa: E731
    p = [cut((0.02 * torch.randn(n + offset, generator=g)).to(pdt)) for n in sizes]
    gr = [cut((1e-3 * torch.randn(n + offset, generator=g)).to(gdt)) for n in sizes]
    m0 = [3e-4 * torch.randn(n, generator=g, dtype=torch.float64).numpy() for n in sizes]
    v0 = [1e-6 * (0.1 + torch.rand(n, generator=g, dtype=torch.float64).numpy()) for n in sizes]
    if bits == 32:
        put = lambda x: cut(torch.cat((torch.zeros(offset), torch.from_numpy(x).float())))  # noqa: E731
        return p, gr, [put(x) for x in m0], [put(x) for x in v0]

    def put8(x, positive):
        c, s, _, _ = ref.encode(x, np.full(len(x), 0.5), positive)
        c = torch.cat((torch.zeros(offset, dtype=torch.uint8), torch.from_numpy(c)))
        return cut(c), torch.from_numpy(s).cuda()

    return p, gr, [put8(x, False) for x in m0], [put8(np.sqrt(x), True) for x in v0]


def state64(s, positive=False):
    if isinstance(s, tuple):
        x = ref.decode(host(s[0]), host(s[1]))
        return x * x if positive else x
    return f64(s)


def moment32(g, m, h):
    """m' in fp32: both products rounded, then their sum."""
    f = np.float32
    b1 = h["betas"][0]
    return (m.astype(f) * f(b1) + g.astype(f) * f(h["grad_scale"]) * f(1 - b1)).astype(np.float64)


def check_step(p, g, m, v, copies=None, decay=None, **over):
    lib = mxq()
    h = {**HYPER, **over}
    r = {k: x for k, x in h.items() if k != "seed"}
    before = [(f64(a), f64(b), state64(c), state64(d, True)) for a, b, c, d in zip(p, g, m, v)]
    lib.AdamW(p, g, m, v, copies, decay).step(**h)
    for j, (a, b, c, d) in enumerate(before):
        if not len(a):
            continue
        wd = r["weight_decay"] * (1.0 if decay is None else decay[j])
        p1, m1, v1, dp, dm, dv = ref.adamw(a, b, c, d, **{**r, "weight_decay": wd})
        half = ref.UBF16 if p[j].dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(f64(p[j]) - p1) <= dp + half * (np.abs(p1) + dp)), j
        if copies is not None and copies[j] is not None:
            assert torch.equal(copies[j], p[j].to(torch.bfloat16)), j
        if not isinstance(m[j], tuple):
            assert np.all(np.abs(f64(m[j]) - m1) <= dm) and np.all(np.abs(f64(v[j]) - v1) <= dv), j
            continue
        um, ur = ref.uniforms(h["seed"], h["step"], j, len(a))
        m32 = moment32(b, c, h)
        assert np.all(np.abs(m32 - m1) <= dm), j
        for (codes, scales), x, u, pos in ((m[j], m32, um, False), (v[j], np.sqrt(v1), ur, True)):
            wc, ws, unsure, near = ref.encode(x, u, pos)
            gc, gs = host(codes), host(scales)
            assert np.array_equal(gs[~near], ws[~near]), j
            sure = ~(unsure | near.repeat(32)[:len(a)])
            assert np.array_equal(gc[sure], wc[sure]), j
            assert sure.mean() > 0.99 or len(a) < 1000
            other = ~sure & ~near.repeat(32)[:len(a)]
            assert np.all(np.abs(gc[other].astype(int) - wc[other].astype(int)) <= 1), j


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(a, b) for a in (torch.float32, torch.bfloat16) for b in (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_step(bits, pdt, gdt, offset):
    p, g, m, v = tensors(SIZES, pdt, gdt, bits, 3, offset)
    check_step(p, g, m, v)
    check_step(p, g, m, v, step=8, seed=2 ** 32 - 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_copies_and_decays(bits):
    p, g, m, v = tensors(SIZES, torch.float32, torch.float32, bits, 4)
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") if i % 3 else None for i, n in enumerate(SIZES)]
    check_step(p, g, m, v, copies, [i % 2 for i in range(len(SIZES))])
    p, g, m, v = tensors([100, 5000], torch.bfloat16, torch.float32, bits, 4)
    check_step(p, g, m, v, [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in (100, 5000)])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_and_empty_tensors(bits):
    sizes = [(37 * i) % 300 for i in range(150)]
    assert 0 in sizes
    p, g, m, v = tensors(sizes, torch.float32, torch.bfloat16, bits, 5)
    check_step(p, g, m, v)
    mxq().AdamW([], [], [], []).step(lr=1.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_states(bits):
    lib = mxq()
    g = torch.Generator().manual_seed(1)
    p, gr = [torch.randn(1000, generator=g).cuda()], [torch.randn(1000, generator=g).cuda()]
    fmt = lib.MXQ_ADAMW_F32 if bits == 32 else lib.MXQ_ADAMW_MXFP8
    check_step(p, gr, [lib.adamw_state(p[0], fmt)], [lib.adamw_state(p[0], fmt)], step=1, grad_scale=1.0)


def test_blocks_of_zeros_and_tiny_values():
    """Zero blocks keep zero scales; values far apart keep their blocks' scales."""
    n = 32 * 6
    p, g, m, v = tensors([n], torch.float32, torch.float32, 8, 6)
    for x in (g[0], m[0][0], v[0][0]):
        x[:64] = 0
    for x in (m[0][1], v[0][1]):
        x[:2] = 0
    g[0][64:96] *= 2.0 ** -30
    g[0][96:128] *= 2.0 ** 40
    for s in (m, v):
        s[0][0][64:96] = 0
        s[0][1][2] = 0
    check_step(p, g, m, v)
    assert host(m[0][1])[0] == 0 and not host(m[0][0])[:32].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_gradients_stay_in_their_elements(bits):
    p, g, m, v = tensors([200], torch.float32, torch.float32, bits, 7)
    q, h, a, b = tensors([200], torch.float32, torch.float32, bits, 7)
    bad = [3, 40, 41, 199]
    g[0][bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")], device="cuda")
    h[0][bad] = 0.0
    lib = mxq()
    lib.AdamW(p, g, m, v).step(**HYPER)
    lib.AdamW(q, h, a, b).step(**HYPER)
    keep = np.setdiff1d(np.arange(200), bad)
    assert np.array_equal(f64(p[0])[keep], f64(q[0])[keep]) and not np.isfinite(f64(p[0])[bad]).any()
    if bits == 8:
        big = {x // 32 for x in bad}  # the largest finite magnitude of such a block may be another one
        same = [i for i in keep if i // 32 not in big]
        assert np.array_equal(host(m[0][0])[same], host(a[0][0])[same])
        assert np.all(np.isnan(state64(m[0])[bad])) and np.all(np.isnan(state64(v[0])[bad]))
        assert np.isfinite(state64(m[0])[keep]).all() and np.isfinite(state64(v[0])[keep]).all()
    else:
        assert not np.isfinite(f64(m[0])[bad]).any() and np.array_equal(f64(m[0])[keep], f64(a[0])[keep])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite_skips_the_step(bits, scale):
    lib = mxq()
    p, g, m, v = tensors([500, 3], torch.float32, torch.float32, bits, 8)
    flat = lambda: [x.clone() for s in (p, m, v) for t in s for x in (t if isinstance(t, tuple) else (t,))]  # noqa: E731
    before = flat()
    opt = lib.AdamW(p, g, m, v)
    opt.step(**{**HYPER, "grad_scale": scale})
    opt.step(**HYPER, control=lib.adamw_control(1e-3, 7, 1, scale))
    opt.step(**HYPER, control=lib.adamw_control(1e-3, 0, 1, 1.0))
    assert all(torch.equal(a, b) for a, b in zip(before, flat()))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 7, 100000])
def test_control_gives_the_same_step(bits, step):
    """lr, scale, step and seed from device memory: the same bits up to the rounding of lr to fp32 (here exact)."""
    lib = mxq()
    h = {**HYPER, "lr": 2.0 ** -10, "step": step}
    a, b = tensors([5000, 77], torch.float32, torch.float32, bits, 9), tensors([5000, 77], torch.float32, torch.float32, bits, 9)
    lib.AdamW(*a).step(**h)
    lib.AdamW(*b).step(**{**h, "lr": 5.0, "step": 3, "grad_scale": 9.0, "seed": 0},
                       control=lib.adamw_control(h["lr"], step, h["seed"], h["grad_scale"]))
    for x, y in zip(a, b):
        for s, t in zip(x, y):
            for u, w in zip(s, t) if isinstance(s, tuple) else ((s, t),):
                assert torch.equal(u, w)


def test_rounding_moves_small_changes():
    """With beta2 = 0.999 one step changes sqrt(v) by far less than half an E4M3 step.  From v = 0 under a constant
    gradient g the stored moments still reach 1 - beta^t of g and g^2: rounding of r by a step of at most r / 8 with the
    probability of its drift leaves a variance of at most r^2 / 8 per element, which the mean of 65536 elements
    does not show, and lifts the mean of r^2 by at most 1/8 of it."""
    lib = mxq()
    n, steps = 1 << 16, 400
    p, g = [torch.zeros(n, device="cuda")], [torch.full((n,), 0.3, device="cuda")]
    m, v = [lib.adamw_state(p[0])], [lib.adamw_state(p[0])]
    opt = lib.AdamW(p, g, m, v)
    for t in range(1, steps + 1):
        opt.step(lr=1e-4, step=t, seed=5)
    assert abs(state64(m[0]).mean() / 0.3 - (1 - 0.9 ** steps)) < 0.02
    want = 0.09 * (1 - 0.999 ** steps)
    assert 0.98 < state64(v[0], True).mean() / want < 1.125


def test_element_past_32_bits():
    """A tensor of more than 2^32 elements: its last blocks, and nothing before them, have gradients."""
    lib = mxq()
    n = (1 << 32) + 100
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = lib.adamw_state(p), lib.adamw_state(p)
    tail = 132  # blocks of 32 counted from the tensor's start
    first = n - tail
    assert first % 32 == 0
    p[first:] = 1.0
    g[first:] = torch.linspace(-1, 1, tail, device="cuda").to(torch.bfloat16)
    big = {"step": 1, "weight_decay": 0.0, "lr": 0.25}  # a step that bf16 parameters of 1 show
    lib.AdamW([p], [g], [m], [v]).step(**{**HYPER, **big})
    p1, m1, v1, dp, _, _ = ref.adamw(np.ones(tail), f64(g[first:]), 0.0, 0.0, **{**REF, **big})
    um, ur = ref.uniforms(HYPER["seed"], 1, 0, tail, first)
    for (codes, scales), x, u, pos in ((m, m1, um, False), (v, np.sqrt(v1), ur, True)):
        wc, ws, unsure, near = ref.encode(x, u, pos)
        sure = ~(unsure | near.repeat(32)[:tail])
        assert np.array_equal(host(scales[first // 32:])[~near], ws[~near])
        assert np.array_equal(host(codes[first:])[sure], wc[sure])
        assert not bool(codes[:first].any()) and not bool(scales[: first // 32].any())
    assert np.all(np.abs(f64(p[first:]) - p1) <= dp + ref.UBF16 * (np.abs(p1) + dp))
    assert not bool(p[:first].any())


def test_on_another_stream():
    lib = mxq()
    a, b = (tensors([5000, 77], torch.float32, torch.float32, 8, 10) for _ in range(2))
    lib.AdamW(*a).step(**HYPER)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lib.AdamW(*b).step(**HYPER, stream=st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) for s, t in ((a[2], b[2]), (a[3], b[3])) for x, y in zip(s, t))


@pytest.mark.parametrize("bits", [32, 8])
def test_places_in_flat_buffers_do_not_matter(bits):
    """The same tensors at other places give the same bits, and nothing beside them is written."""
    m = mxq()
    p, g, mm, vv = tensors(SIZES, torch.float32, torch.float32, bits, 9)
    flat = lambda x: [x] if torch.is_tensor(x) else list(x)  # noqa: E731
    groups = [p, g, [flat(x)[0] for x in mm], [flat(x)[0] for x in vv]]
    for shifts in ((1, 1, 1, 1), (31, 31, 31, 31), (5, 2, 30, 17), (0, 3, 32, 64)):
        placed, beside = [], []
        for xs, o in zip(groups, shifts):
            guard = 77 if xs[0].dtype == torch.uint8 else -7.5
            buf = torch.full((sum(len(x) + 3 for x in xs) + o + 40,), guard, dtype=xs[0].dtype, device="cuda")
            free, views = torch.ones(len(buf), dtype=torch.bool, device="cuda"), []
            for x in xs:
                buf[o:o + len(x)] = x
                free[o:o + len(x)] = False
                views.append(buf[o:o + len(x)])
                o += len(x) + 3
            placed.append(views)
            beside.append((buf, free, guard))
        scales = lambda s: [x[1].clone() for x in s]  # noqa: E731
        a = [[x.clone() for x in xs] for xs in groups]
        am, av, bm, bv = a[2], a[3], placed[2], placed[3]
        if bits == 8:
            am, av = list(zip(am, scales(mm))), list(zip(av, scales(vv)))
            bm, bv = list(zip(bm, scales(mm))), list(zip(bv, scales(vv)))
        for args in ((a[0], a[1], am, av), (placed[0], placed[1], bm, bv)):
            m.AdamW(*args).step(step=3, seed=11)
        for one, other in zip(a, placed):
            assert all(torch.equal(x, y) for x, y in zip(one, other)), shifts
        for buf, free, guard in beside:
            assert torch.all(buf[free] == guard), shifts


@pytest.mark.parametrize("bits", [32, 8])
def test_the_least_eps_leaves_untouched_elements(bits):
    """Elements without gradient or state stay where they are under the smallest eps that is accepted."""
    lib = mxq()
    fmt = lib.MXQ_ADAMW_F32 if bits == 32 else lib.MXQ_ADAMW_MXFP8
    p = torch.linspace(-1, 1, 300, device="cuda")
    want, m, v = p.clone(), lib.adamw_state(p, fmt), lib.adamw_state(p, fmt)
    lib.AdamW([p], [torch.zeros_like(p)], [m], [v]).step(lr=0.1, eps=2.0 ** -126, weight_decay=0.0)
    assert torch.equal(p, want)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr", [float("nan"), float("inf")])
def test_a_control_rate_that_is_not_finite_skips_the_step(bits, lr):
    """As the config's own rate is refused."""
    lib = mxq()
    p, g, m, v = tensors([500, 3], torch.float32, torch.float32, bits, 8)
    flat = lambda: [x.clone() for s in (p, m, v) for t in s for x in (t if isinstance(t, tuple) else (t,))]  # noqa: E731
    before = flat()
    lib.AdamW(p, g, m, v).step(**HYPER, control=lib.adamw_control(lr, 7, 1, 1.0))
    assert all(torch.equal(a, b) for a, b in zip(before, flat()))


def near_the_border(u, e, rng):
    """E4M3 values + (1 - u +- 2^-18) of their step, times 2^e, each an fp32 number from 2^-6 to below 448 before the 2^e:
    rounded up with the plus and down with the minus."""
    k = rng.integers(8, 126, len(u))  # normal codes with a successor
    up = rng.integers(0, 2, len(u)).astype(bool)
    y = ref.E4M3[k] + (1 - u + np.where(up, 2.0 ** -18, -(2.0 ** -18))) * (ref.E4M3[k + 1] - ref.E4M3[k])
    x = y * 2.0 ** e
    assert np.array_equal(x.astype(np.float32).astype(np.float64), x)
    return x, np.where(up, k + 1, k)


@pytest.mark.parametrize("values", ["near the border", "of E4M3"])
@pytest.mark.parametrize("moment", ["m", "r"])
def test_rounding_is_decided_within_2_to_the_minus_18_of_a_step(moment, values):
    """Under every scale; values that E4M3 holds keep their codes.  With betas of 0, m' is the gradient and r its
    magnitude, both exactly."""
    lib = mxq()
    rng = np.random.default_rng(5)
    lo, hi = (-110, 110) if moment == "m" else (-50, 55)  # squares stay normal
    exps = np.repeat(np.arange(lo, hi), 32)
    n = 32 * len(exps)
    um, ur = ref.uniforms(77, 3, 0, n)
    if values == "of E4M3":
        code = rng.integers(1, 127, n)
        x = ref.E4M3[code] * 2.0 ** exps.repeat(32)
    else:
        x, code = near_the_border(um if moment == "m" else ur, exps.repeat(32).astype(np.float64), rng)
    x[::32], code[::32] = 448.0 * 2.0 ** exps, 126  # fixes the block's scale
    p, g = torch.zeros(n, device="cuda"), torch.from_numpy(x.astype(np.float32)).cuda()
    m, v = lib.adamw_state(p), lib.adamw_state(p)
    lib.AdamW([p], [g], [m], [v]).step(lr=0.0, betas=(0.0, 0.0), weight_decay=0.0, step=3, seed=77)
    codes, scales = m if moment == "m" else v
    assert np.array_equal(host(scales), (exps + 127).astype(np.uint8))
    assert np.array_equal(host(codes), code.astype(np.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [47, 50, 51, 64, 101])
def test_as_many_tensors_as_a_launch_holds_and_more(bits, count):
    p, g, m, v = tensors([1 + 37 * i % 90 for i in range(count)], torch.bfloat16, torch.float32, bits, count)
    check_step(p, g, m, v)
