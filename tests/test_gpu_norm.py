"""The residual norm on the GPU against its formulas in float64.

Tolerances (relative L2; per element see updater_oracle.check), u = unit roundoff of the type, v that of float32:
- y: one rounding to the type, and in float32 the sum (its two roundings, h), the mean of squares (terms of one sign, added
  in chains of at most 32 and a tree of 10: half of sqrt(42) v in the root), the root, the division and two products:
  10 v; 16 v are allowed.
- gradients of x and the residual: one rounding to the type, the root and c as above, four products and sums: 24 v.
- gradient of the weight: 16 v for the factors and 2 sqrt(K) v for a sum of K rows, and the rounding to its type.
- 8-bit codes: half a step, 2^-4 of the value or half of the smallest step 2^-9, times the scale; scales 16 v.
"""
import math

import pytest
import torch

import updater_oracle as o

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
V = 2.0 ** -24
EPS = 1e-6


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def randn(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def inputs(rows, width, dtype, stream, seed=0, wdtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (randn(g, rows, width, dtype=dtype), randn(g, rows, width, scale=3, dtype=stream),
            (1 + randn(g, width, scale=0.1)).to(wdtype), randn(g, rows, width, dtype=dtype),
            randn(g, rows, width, dtype=stream))


def reference(x, residual, w):
    h = x.double() + (residual.double() if residual is not None else 0)
    return h, h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w.double()


def reference_grads(h, w, dy, dh):
    h, w, dy = h.double(), w.double(), dy.double()
    inv = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    n, u = h * inv, dy * w
    d = inv * (u - n * (u * n).mean(1, keepdim=True))
    return d + (dh.double() if dh is not None else 0), (dy * n).sum(0)


def rel(dtype, v):
    return v * V + (o.UNIT[dtype] if dtype != torch.float32 else 0)


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 33), (17, 128), (16, 129), (9, 256), (33, 500), (64, 512), (7, 513), (48, 1024),
          (5, 1025), (4, 2048), (3, 2049), (3, 8191), (2, 8192), (2, 8193), (3, 20001)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("wide_stream", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(shape, wide_stream, dtype):
    rows, width = shape
    stream = torch.float32 if wide_stream else dtype
    wdtype = dtype if width % 2 else torch.float32
    x, residual, w, dy, dh = inputs(rows, width, dtype, stream, wdtype=wdtype)
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    y, h = norm.forward(x, residual)
    rh, ry = reference(x, residual, w)
    o.check(y, ry, rel(dtype, 16), "y")
    o.check(h, rh, rel(stream, 1), "h")
    got = norm.backward(h, dy, dh)
    d, dw = reference_grads(h, w, dy, dh)
    o.check(got["x"], d, rel(dtype, 24), "x")
    o.check(got["residual"], d, rel(stream, 24), "residual")
    o.check(got["weight"], dw, rel(wdtype, 16 + 2 * math.sqrt(rows)), "weight")
    assert got["weight"].dtype == wdtype and got["residual"].dtype == stream
    for k, v in norm.backward(h, dy, dh).items():
        assert torch.equal(v, got[k]), k


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(70000, 100), (20011, 512), (9001, 1000), (3000, 3000), (300, 9000)], ids=str)
def test_many_rows(shape, dtype):
    """More rows than the workgroups hold at once."""
    rows, width = shape
    x, residual, w, dy, dh = inputs(rows, width, dtype, torch.float32, seed=1)
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    y, h = norm.forward(x, residual)
    rh, ry = reference(x, residual, w)
    o.check(y, ry, rel(dtype, 16), "y")
    o.check(h, rh, V, "h")
    got = norm.backward(h, dy, dh)
    d, dw = reference_grads(h, w, dy, dh)
    o.check(got["x"], d, rel(dtype, 24), "x")
    o.check(got["residual"], d, 24 * V, "residual")
    o.check(got["weight"], dw, (16 + 2 * math.sqrt(rows)) * V, "weight")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_without_residual_and_dh(dtype):
    x, _, w, dy, _ = inputs(37, 200, dtype, dtype, seed=2)
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    y, h = norm.forward(x)
    assert h is x
    o.check(y, reference(x, None, w)[1], rel(dtype, 16), "y")
    start = torch.empty(37, 200, device="cuda")
    y2, h2 = norm.forward(x, h=start)
    assert h2 is start and torch.equal(start, x.float()) and torch.equal(y, y2)
    only = {"weight": torch.empty_like(w)}
    assert set(norm.backward(x, dy, grads=only)) == {"weight"}
    d, dw = reference_grads(x, w, dy, None)
    o.check(only["weight"], dw, (16 + 2 * math.sqrt(37)) * V, "weight")
    o.check(norm.backward(x, dy, grads={"x": torch.empty_like(x)})["x"], d, rel(dtype, 24), "x")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("width", [61, 700, 2500, 9000])
def test_strides_and_alignment(width, dtype):
    """Rows of odd strides that start at odd elements; what lies between the rows is left alone."""
    x, residual, w, dy, dh = inputs(11, width, dtype, dtype, seed=3, wdtype=dtype)
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    y, h = norm.forward(x, residual)
    grads = norm.backward(h, dy, dh)

    def spread(t, gap, fill=7.0):
        wide = torch.full((t.shape[0], width + gap), fill, dtype=t.dtype, device="cuda")
        view = wide[:, 1:width + 1]
        view.copy_(t)
        return wide, view

    views = [spread(t, 2 + k)[1] for k, t in enumerate((x, residual, h, dy, dh))]
    wy, vy = spread(torch.zeros_like(y), 5)
    wh, vh = spread(torch.zeros_like(h), 3)
    wx, vx = spread(torch.zeros_like(x), 9)
    norm.forward(views[0], views[1], y=vy, h=vh)
    norm.backward(views[2], views[3], views[4], grads={"x": vx})
    for wide, view, want in ((wy, vy, y), (wh, vh, h), (wx, vx, grads["x"])):
        assert torch.equal(view, want)
        assert (wide[:, 0] == 7).all() and (wide[:, width + 1:] == 7).all()


@pytest.mark.parametrize("width", [96, 1500, 9000])
def test_in_place(width):
    dtype = torch.bfloat16
    x, residual, w, dy, dh = inputs(301, width, dtype, torch.float32, seed=4)
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    y, h = norm.forward(x, residual)
    g = norm.backward(h, dy, dh, grads={"x": torch.empty_like(x), "residual": torch.empty_like(residual)})
    x2, r2 = x.clone(), residual.clone()
    y2, h2 = norm.forward(x2, r2, y=x2, h=r2)
    assert y2 is x2 and h2 is r2 and torch.equal(x2, y) and torch.equal(r2, h)
    norm.backward(h, dy, dh, grads={"x": dy, "residual": dh})
    assert torch.equal(dy, g["x"]) and torch.equal(dh, g["residual"])


def check_codes(codes, scales, y, group):
    rows, width = y.shape
    group = group or width
    parts = torch.nn.functional.pad(y, (0, -width % group)).view(rows, -1, group)
    top = parts.abs().amax(2)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert scales.shape == want.shape
    assert ((scales.double() - want).abs() <= 16 * V * want).all()
    got = torch.nn.functional.pad(codes.double(), (0, -width % group)).view(rows, -1, group) * scales.double()[..., None]
    off = (got - parts).abs()
    # half a step, and the scale's and y's own errors, which may carry a value over a border between two codes
    assert (off <= (2.0 ** -4 + 64 * V) * parts.abs() + (2.0 ** -10 + 64 * V) * want[..., None]).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (5, 31), (17, 128), (9, 300), (33, 512), (6, 1000), (3, 2100), (2, 9000)],
                         ids=str)
def test_8bit(shape, group, dtype):
    rows, width = shape
    x, residual, w, _, _ = inputs(rows, width, dtype, dtype, seed=5)
    x[0], residual[0] = 0, 0          # a row of zeros
    residual[rows - 1, ::3] *= 1e-3   # codes below the normal range
    norm = gsr().ResidualNorm(w, dtype, eps=EPS)
    codes, scales, h = norm.forward8(x, residual, group=group)
    rh, ry = reference(x, residual, w)
    o.check(h, rh, rel(dtype, 1), "h")
    assert codes.dtype == torch.float8_e4m3fn
    check_codes(codes, scales, ry, group)
    assert (codes[0].float() == 0).all() and (scales[0] == 1).all()


def test_8bit_tiny_values():
    """Values whose scale is not a normal float32's reciprocal away from overflow."""
    w = torch.full((64,), 1e-36, device="cuda")
    x = inputs(3, 64, torch.float32, torch.float32, seed=6)[0]
    codes, scales, _ = gsr().ResidualNorm(w, torch.float32, eps=EPS).forward8(x)
    check_codes(codes, scales, reference(x, None, w)[1], 0)


@pytest.mark.parametrize("width", [100, 1000, 5000, 9000])
def test_infinities_stay_in_their_row(width):
    x, residual, w, dy, dh = inputs(8, width, torch.float32, torch.float32, seed=7)
    norm = gsr().ResidualNorm(w, torch.float32, eps=EPS)
    y, h = norm.forward(x, residual)
    g = norm.backward(h, dy, dh)
    x[2, 5], x[4, width - 1] = float("inf"), float("nan")
    y2, h2 = norm.forward(x, residual)
    g2 = norm.backward(h2, dy, dh)
    c2, s2, _ = norm.forward8(x, residual)
    keep = [0, 1, 3, 5, 6, 7]
    assert torch.equal(y2[keep], y[keep]) and torch.equal(g2["x"][keep], g["x"][keep])
    assert torch.isnan(y2[4]).all() and torch.isnan(y2[2, 5])
    assert torch.isfinite(s2[keep]).all() and torch.isfinite(c2[keep].float()).all()


def test_no_rows():
    w = torch.ones(40, device="cuda")
    norm = gsr().ResidualNorm(w, torch.bfloat16)
    x = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    y, h = norm.forward(x, x)
    g = norm.backward(x, x)
    assert y.shape == (0, 40) and (g["weight"] == 0).all()
    codes, scales, _ = norm.forward8(x, group=32)
    assert codes.shape == (0, 40) and scales.shape == (0, 2)


def test_gradients_against_differences():
    """Central differences of the forward pass along random directions, float32; the difference's own rounding is
    16 V |L| / step and its truncation step^2, with a step of 1e-2: 1e-4 of the gradient's size and to spare."""
    x, residual, w, dy, dh = inputs(6, 90, torch.float32, torch.float32, seed=8)
    norm = gsr().ResidualNorm(w, torch.float32, eps=EPS)
    _, h = norm.forward(x, residual)
    g = norm.backward(h, dy, dh)

    def loss(x, w):
        y, h = gsr().ResidualNorm(w, torch.float32, eps=EPS).forward(x, residual)
        return (y.double() * dy.double()).sum() + (h.double() * dh.double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(9)
    for name, at in (("x", x), ("weight", w)):
        d = torch.randn(at.shape, generator=gen, device="cuda")
        step = 1e-2
        up = loss(x + step * d, w) if name == "x" else loss(x, w + step * d)
        down = loss(x - step * d, w) if name == "x" else loss(x, w - step * d)
        slope = (g[name].double() * d.double()).sum()
        assert abs((up - down) / (2 * step) - slope) <= 1e-3 * g[name].double().norm() * d.double().norm()


def test_streams_and_graph():
    x, residual, w, dy, dh = inputs(500, 512, torch.bfloat16, torch.float32, seed=10)
    norm = gsr().ResidualNorm(w, torch.bfloat16, eps=EPS)
    y, h = norm.forward(x, residual)
    g = norm.backward(h, dy, dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, h2 = norm.forward(x, residual, stream=side)
    g2 = norm.backward(h2, dy, dh, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, h3 = norm.forward(x, residual)
        g3 = norm.backward(h3, dy, dh)
    for seed in (11, 12, 13):
        new = inputs(500, 512, torch.bfloat16, torch.float32, seed=seed)
        for t, s in zip((x, residual, dy, dh), (new[0], new[1], new[3], new[4])):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        y, h = norm.forward(x, residual)
        g = norm.backward(h, dy, dh)
        assert torch.equal(y, y3) and torch.equal(h, h3) and all(torch.equal(g[k], g3[k]) for k in g)


def test_refusals():
    w = torch.ones(16, device="cuda")
    m = gsr()
    norm = m.ResidualNorm(w, torch.bfloat16)
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        m.ResidualNorm(w.double(), torch.float32)
    with pytest.raises(ValueError):
        m.ResidualNorm(w.half(), torch.bfloat16)
    with pytest.raises(ValueError):
        norm.forward(x.float())
    with pytest.raises(ValueError):
        norm.forward(x, x.half())
    with pytest.raises(ValueError):
        norm.forward(x.t().contiguous().t())
    with pytest.raises(ValueError):
        norm.forward8(x, group=16)
    with pytest.raises(m.GsrError):
        m.ResidualNorm(w, torch.bfloat16, eps=-1.0).forward(x)
    wide = torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.GsrError):
        norm.forward(wide[:4], y=wide[1:])
    with pytest.raises(m.GsrError):
        norm.forward(x, x, y=x)


def test_8bit_rows_with_infinities():
    """Codes of the y that the formula gives: NaN through the row of a NaN; zeros beside an infinity, NaN in its place."""
    x = inputs(3, 300, torch.float32, torch.float32, seed=14)[0]
    x[0, 40], x[1, 70] = float("nan"), float("inf")
    for group in (0, 32):
        codes, scales, _ = gsr().ResidualNorm(torch.ones(300, device="cuda"), torch.float32, eps=EPS).forward8(x, group=group)
        codes = codes.float()
        assert torch.isnan(codes[0]).all() and torch.isnan(codes[1, 70])
        rest = torch.arange(300, device="cuda") != 70
        assert (codes[1, rest] == 0).all() and (scales[:2] == 1).all() and torch.isfinite(codes[2]).all()


@pytest.mark.parametrize("group", [0, 32])
def test_8bit_subnormal_values(group):
    """Beside a code's half step: a scale rounded among the subnormal numbers, 2^-150 for each of up to 448 of them."""
    x = torch.full((6, 96), 1e-36, device="cuda") * torch.linspace(-1, 1, 96, device="cuda")
    w = torch.full((96,), 1.0, device="cuda")
    for k, size in enumerate((1.0, 1e-4, 1e-6, 1e-8, 1e-9, 1e-12)):
        codes, scales, _ = gsr().ResidualNorm(w * size, torch.float32, eps=EPS).forward8(x, group=group)
        y = x.double() / math.sqrt(EPS) * (w * size).double()
        s = scales.double().repeat_interleave(group or 96, 1)
        err = (codes.double() * s - y).abs()
        assert (err <= (2.0 ** -4 + 32 * V) * y.abs() + (2.0 ** -10 + 32 * V) * s + 448 * 2.0 ** -150).all(), k
