"""The AdamW step on the GPU against its formulas in float64.

Tolerances, V = 2^-24: m and v are two products and a sum (with the coefficients' own roundings 5 V of the terms); the step
divides them (their error, a root, two products, a division, the two corrections: 12 V of |lr m / c1| / (...) taken with the
terms of m), and the parameter is rounded once.  8-bit states: half a step, 2^-4 of the value or 2^-10 of the scale, and 16 V
of the scale for its own error.  16-bit parameters and copies: one rounding.
"""
import math

import pytest
import torch

import updater_oracle as o

pytestmark = pytest.mark.gpu
V = 2.0 ** -24
BETAS, EPS = (0.9, 0.999), 1e-8


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def make(sizes, dtype=torch.float32, gdtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ps = [torch.randn(s, generator=gen, device="cuda").to(dtype) for s in sizes]
    gs = []
    for s in sizes:
        g = torch.randn(s, generator=gen, device="cuda") * torch.exp(2 * torch.randn(s, generator=gen, device="cuda"))
        gs.append((g * (torch.rand(s, generator=gen, device="cuda") > 0.2)).to(gdtype))
    return ps, gs


def held(opt, i):
    """(m, v) of tensor i in float64, as the states stand for them."""
    if not opt.m_scale:
        return opt.m[i].double(), opt.v[i].double()
    n = opt.m[i].numel()
    m = opt.m[i].double() * opt.m_scale[i].double().repeat_interleave(256)[:n]
    return m, (opt.v[i].double() * opt.v_scale[i].double().repeat_interleave(256)[:n]) ** 2


def expected(p, g, m, v, t, lr, wd, gs=1.0):
    """New p, m, v in float64, and what their errors are relative to."""
    p, g = p.double().flatten(), g.double().flatten() * gs
    b1, b2 = BETAS
    terms = (b1 * m).abs() + ((1 - b1) * g).abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    down = torch.sqrt(v / (1 - b2 ** t)) + EPS
    step = lr * m / (1 - b1 ** t) / down
    return p - lr * wd * p - step, m, v, terms, lr * terms / (1 - b1 ** t) / down


def check_codes(codes, scales, want, root):
    blocks = torch.nn.functional.pad(want, (0, -want.numel() % 256)).view(-1, 256)
    top = blocks.abs().amax(1)
    scale = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert ((scales.double() - scale).abs() <= 32 * V * scale).all()
    s = scales.double().repeat_interleave(256)[:want.numel()]
    got = codes.double() * s
    allowed = (2.0 ** -4 + 64 * V) * want.abs() + (2.0 ** -10 + 64 * V) * s
    if root:  # a value above zero is at least the smallest code
        assert (got[want > 0] > 0).all()
        allowed = torch.where((want > 0) & (want < s * 2.0 ** -9), s * 2.0 ** -9, allowed)
    assert ((got - want).abs() <= allowed).all()


SIZES = [(1,), (3, 5), (256,), (257,), (4095,), (4097,), (50, 3), (20000, 3), (1000, 16, 3), (7,), (100003,)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype, gdtype, cdtype", [
    (torch.float32, torch.float32, None), (torch.float32, torch.bfloat16, torch.bfloat16),
    (torch.float32, torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16, None),
    (torch.float16, torch.float32, torch.float32)], ids=str)
def test_steps(dtype, gdtype, cdtype, bits):
    ps, _ = make(SIZES, dtype)
    copies = [torch.empty(p.shape, dtype=cdtype, device="cuda") for p in ps] if cdtype else None
    lr = [1e-3 * (1 + k) for k in range(len(SIZES))]
    wd = [0.0 if k % 2 else 0.1 for k in range(len(SIZES))]
    opt = gsr().AdamW(ps, lr=lr, betas=BETAS, eps=EPS, weight_decay=wd, state_bits=bits, copies=copies)
    for t in range(1, 5):
        _, grads = make(SIZES, dtype, gdtype, seed=t)
        before = [(p.clone(), *held(opt, i)) for i, p in enumerate(ps)]
        opt.step(grads)
        assert int(opt.steps) == t
        for i, (p, m, v) in enumerate(before):
            want, wm, wv, terms, move = expected(p, grads[i], m, v, t, lr[i], wd[i])
            u = V if dtype == torch.float32 else o.UNIT[dtype]
            got = ps[i].double().flatten()
            tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
            assert ((got - want).abs() <= u * want.abs() + 4 * V * p.double().flatten().abs() + 32 * V * move + tiny).all(), i
            if cdtype:
                c = copies[i].double().flatten()
                cu = V if cdtype == torch.float32 else o.UNIT[cdtype]
                low = 2.0 ** -25 if cdtype == torch.float16 else 0.0
                assert ((c - want).abs() <= cu * want.abs() + 8 * V * p.double().flatten().abs() + 32 * V * move + low).all()
            if bits == 32:
                assert ((opt.m[i].double() - wm).abs() <= 5 * V * terms).all()
                assert ((opt.v[i].double() - wv).abs() <= 5 * V * wv + 1e-44).all()
            else:
                check_codes(opt.m[i], opt.m_scale[i], wm, False)
                check_codes(opt.v[i], opt.v_scale[i], wv.sqrt(), True)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More tensors than one launch holds, some without a gradient, some empty: the same as each by itself."""
    sizes = [((37 * k) % 700,) for k in range(130)]
    ps, gs = make(sizes)
    alone = [p.clone() for p in ps]
    gs = [None if k % 11 == 3 else g for k, g in enumerate(gs)]
    opt = gsr().AdamW(ps, lr=0.01, weight_decay=0.1, state_bits=bits)
    for _ in range(2):
        opt.step(gs)
    assert int(opt.steps) == 2
    for k, (p, g) in enumerate(zip(alone, gs)):
        if g is not None and p.numel():
            one = gsr().AdamW([p], lr=0.01, weight_decay=0.1, state_bits=bits)
            one.step([g])
            one.step([g])
        assert torch.equal(p, ps[k]), k


def test_unaligned_views():
    flat, gflat = (torch.randn(5000, generator=torch.Generator(device="cuda").manual_seed(s), device="cuda") for s in (1, 2))
    keep = flat.clone()
    ps = [flat[1:1002], flat[1003:1003 + 2000].view(20, 100)]
    gs = [gflat[3:1004], gflat[1501:3501].view(20, 100)]
    ref = [p.clone() for p in ps]
    gsr().AdamW(ref, lr=0.1).step([g.clone() for g in gs])
    gsr().AdamW(ps, lr=0.1).step(gs)
    assert all(torch.equal(a, b) for a, b in zip(ps, ref))
    for lo, hi in ((0, 1), (1002, 1003), (3003, 5000)):
        assert torch.equal(flat[lo:hi], keep[lo:hi])


def test_scales_on_the_device():
    """Gradients and rates times scalars that are read at the time of the step."""
    ps, gs = make([(1000,), (64, 3)], seed=3)
    ref = [p.clone() for p in ps]
    gsr().AdamW(ref, lr=0.01 * 0.5, weight_decay=0.1).step([g * 0.25 for g in gs])
    scale, rate = torch.tensor([0.25], device="cuda"), torch.tensor(0.5, device="cuda")
    gsr().AdamW(ps, lr=0.01, weight_decay=0.1).step(gs, grad_scale=scale, rate_scale=rate)
    for p, r in zip(ps, ref):
        assert ((p - r).abs() <= 16 * V * r.abs() + 32 * V * 0.01).all()


def test_zero_gradients_do_not_explode():
    """A root that is tiny next to its block's largest keeps m / sqrt(v) in bounds when the gradients stop."""
    p = torch.zeros(256, device="cuda")
    opt = gsr().AdamW([p], lr=1.0, state_bits=8)
    g = torch.full((256,), 1e-8, device="cuda")
    g[0] = 1.0
    opt.step([g])
    for _ in range(5):
        before = p.clone()
        opt.step([torch.zeros_like(g)])
        # |m / c1| / sqrt(v / c2) with both held: at most a code's error over what the exact step gives
        assert (p - before).abs().max() <= 10.0


def test_not_a_number_stays_in_its_block():
    p, g = torch.ones(1024, device="cuda"), torch.full((1024,), 0.1, device="cuda")
    g[300] = float("nan")
    opt = gsr().AdamW([p], lr=0.1, state_bits=8)
    opt.step([g])
    opt.step([torch.full_like(g, 0.1)])
    assert torch.isfinite(p[:256]).all() and torch.isfinite(p[512:]).all() and torch.isnan(p[300])


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_counts_on(bits):
    sizes = [(5000,), (33, 7)]
    ps, gs = make(sizes, seed=4)
    ref = [p.clone() for p in ps]
    opt, other = (gsr().AdamW(x, lr=0.01, weight_decay=0.01, state_bits=bits) for x in (ps, ref))
    grads = [torch.zeros_like(g) for g in gs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads)
    assert int(opt.steps) == 0
    for k in range(4):
        _, new = make(sizes, seed=10 + k)
        for a, n in zip(grads, new):
            a.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        other.step(new)
        assert int(opt.steps) == int(other.steps) == k + 1
        assert all(torch.equal(a, c) for a, c in zip(ps, ref))


def test_another_stream():
    ps, gs = make([(70000,)], seed=5)
    ref = [p.clone() for p in ps]
    a, c = gsr().AdamW(ps, lr=0.01), gsr().AdamW(ref, lr=0.01)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.step(gs, stream=side)
        c.step(gs)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ps[0], ref[0])


def test_follows_a_quadratic():
    """|x - target|^2 falls to the step's size from any start: the corrections and signs together."""
    target = torch.linspace(-1, 1, 1000, device="cuda")
    for bits in (32, 8):
        x = torch.zeros(1000, device="cuda")
        opt = gsr().AdamW([x], lr=0.02, state_bits=bits)
        for _ in range(300):
            opt.step([2 * (x - target)])
        assert (x - target).abs().max() < 0.1


def test_refusals():
    m = gsr()
    p, g = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    for bad in (lambda: m.AdamW([]), lambda: m.AdamW([p], state_bits=16), lambda: m.AdamW([p], lr=[1.0, 2.0]),
                lambda: m.AdamW([p.double()]), lambda: m.AdamW([torch.zeros(4, 4, device="cuda").t()[:2]]),
                lambda: m.AdamW([p], copies=[torch.zeros(99, device="cuda")]), lambda: m.AdamW([p]).step([g[:50]]),
                lambda: m.AdamW([p]).step([g, g]), lambda: m.AdamW([p]).step([g.double()]),
                lambda: m.AdamW([p]).step([g.cpu()]),
                lambda: m.AdamW([p]).step([g], grad_scale=torch.ones(1, device="cuda").double())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.AdamW([p, p]).step([g, g]), lambda: m.AdamW([p]).step([p]),
                lambda: m.AdamW([p], copies=[g]).step([g]), lambda: m.AdamW([p], betas=(1.0, 0.9)).step([g]),
                lambda: m.AdamW([p], eps=0.0).step([g]), lambda: m.AdamW([p], lr=float("nan")).step([g])):
        with pytest.raises(m.GsrError):
            bad()
    assert (p == 0).all()


def test_states_that_fade():
    """Without gradients m falls by b1 a step, through the subnormal numbers, where a scale could be rounded to nothing."""
    p = torch.zeros(600, device="cuda")
    opt = gsr().AdamW([p], lr=1.0, state_bits=8)
    g = torch.full((600,), 1e-36, device="cuda") * torch.linspace(-1, 1, 600, device="cuda")
    opt.step([g])
    for _ in range(250):
        m, v = held(opt, 0)
        opt.step([torch.zeros_like(g)])
        s = opt.m_scale[0].double().repeat_interleave(256)[:600]
        assert (opt.m_scale[0] >= 2.0 ** -126).all() and torch.isfinite(p).all()
        err = (held(opt, 0)[0] - 0.9 * m).abs()
        assert (err <= (2.0 ** -4 + 64 * V) * 0.9 * m.abs() + (2.0 ** -10 + 64 * V) * s + 2.0 ** -149).all()
    # the least scale's smallest codes round to themselves: 0.9 k is within half of k up to 5
    assert (held(opt, 0)[0].abs() <= 5 * 2.0 ** -9 * 2.0 ** -126).all()
