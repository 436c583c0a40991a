"""The updater's operators on the GPU against their float64 definitions.

Tolerances (relative L2; per element see updater_oracle.check), u = unit roundoff of the type:
- block, 16-bit: every rounding to the type on the way to a result counts one u -- y: h, y (2 u); w_down: h, w_down
  (2 u); x, w_gate, w_up: g, u, dg or du, the result (4 u).  float32: split products leave out 2^-24 of each
  product and a sum of K terms in float32 loses at most about sqrt(K) u, over the two or three products in a row:
  16 u + 2 sqrt(K) u with K the longest sum.
- recurrence: one rounding for 16-bit results (1 u); float32: the sigmoid's few u, kept over the state's memory of at
  most 1 / (1 - a): 32 u.  The states stay float32 in every type.
- orthogonalisation, bfloat16 result: 15 roundings of X, P, Q to 2^-12 and one to 2^-9; float32: 15 to 2^-22, doubled
  for the left-out lo lo products.
"""
import math

import numpy as np
import pytest
import torch

import updater_oracle as o

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def randn(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def ffn_inputs(m, d, f, out, dtype, seed=0):
    g = gen(seed)
    return (randn(g, m, d, dtype=dtype), randn(g, f, d, scale=d ** -0.5, dtype=dtype),
            randn(g, f, d, scale=d ** -0.5, dtype=dtype), randn(g, out, f, scale=f ** -0.5, dtype=dtype),
            randn(g, m, out, dtype=dtype))


def ffn_tol(dtype, roundings, k):
    u = o.UNIT[dtype]
    return roundings * u if dtype != torch.float32 else (16 + 2 * math.sqrt(k)) * u


SHAPES = [(1, 1, 1, 1), (1, 64, 96, 48), (2, 8, 8, 8), (16, 72, 40, 24), (17, 57, 131, 33), (63, 128, 64, 256),
          (64, 100, 300, 61), (65, 33, 257, 40), (129, 64, 65, 66), (300, 200, 136, 72), (1000, 57, 256, 128)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ffn(shape, act, dtype):
    m, d, f, out = shape
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, dtype)
    block = gsr().GatedFFN(wg, wu, wd, activation=act)
    y = block.forward(x)
    y2, saved = block.forward(x, save=True)
    got = block.backward(x, saved, dy)
    torch.cuda.synchronize()
    ref = o.ffn(x, wg, wu, wd, act, dy)
    k = max(m, 2 * f, d, out)
    o.check(y, ref["y"], ffn_tol(dtype, 2, k), "y")
    o.check(y2, ref["y"], ffn_tol(dtype, 2, k), "y of the saving pass")
    o.check(got["w_down"], ref["w_down"], ffn_tol(dtype, 2, k), "w_down")
    for name in ("x", "w_gate", "w_up"):
        o.check(got[name], ref[name], ffn_tol(dtype, 4, k), name)


@pytest.mark.parametrize("dtype, shape", [(torch.bfloat16, (25000, 256, 520, 264)), (torch.float16, (9000, 512, 1366, 520)),
                                          (torch.float32, (20000, 57, 256, 128))], ids=str)
def test_ffn_large_tiles_and_split_gradients(dtype, shape):
    """Enough rows for the large tiles, and weight gradients split along them."""
    m, d, f, out = shape
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, dtype, seed=3)
    block = gsr().GatedFFN(wg, wu, wd, activation="gelu")
    y, saved = block.forward(x, save=True)
    got = block.backward(x, saved, dy)
    ref = o.ffn(x, wg, wu, wd, "gelu", dy)
    o.check(y, ref["y"], ffn_tol(dtype, 2, m), "y")
    o.check(got["w_down"], ref["w_down"], ffn_tol(dtype, 2, m), "w_down")
    for name in ("x", "w_gate", "w_up"):
        o.check(got[name], ref[name], ffn_tol(dtype, 4, m), name)
    again = block.backward(x, saved, dy)
    for name in got:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("shape, act", [((33000, 200, 520, 193), "silu"), ((2100, 1024, 1366, 1024), "gelu"),
                                        ((70001, 256, 250, 192), "gelu"), ((70000, 120, 500, 130), "silu")], ids=str)
def test_ffn_float32_large(shape, act):
    """float32 products large enough to run on split operands, or (narrow rows) on large tiles of the float32 ones; one
    NaN and one infinite row, strided x."""
    m, d, f, out = shape
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, torch.float32, seed=8)
    wide = torch.zeros(m, d + 3, device="cuda")
    wide[:, 1:d + 1] = x
    xv = wide[:, 1:d + 1]
    block = gsr().GatedFFN(wg, wu, wd, activation=act)
    y, saved = block.forward(xv, save=True)
    got = block.backward(xv, saved, dy)
    ref = o.ffn(x, wg, wu, wd, act, dy)
    tol = ffn_tol(torch.float32, 0, max(m, 2 * f, d, out))
    o.check(y, ref["y"], tol, "y")
    assert torch.equal(block.forward(xv), y)
    for name in ("w_down", "x", "w_gate", "w_up"):
        o.check(got[name], ref[name], tol, name)
    xv[130, 7], xv[m - 1, d - 1] = float("nan"), float("inf")
    bad = block.forward(xv)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[[130, m - 1]] = False
    assert torch.equal(bad[keep], y[keep]) and torch.isnan(bad[130]).all() and not torch.isfinite(bad[m - 1]).any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("off", [0, 1, 3])
def test_ffn_strides_and_alignment(dtype, off):
    """Row views of wider arrays, starting off any 16-byte boundary, for inputs and outputs; guard columns intact."""
    m, d, f, out = 70, 64, 72, 40
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, dtype, seed=4)

    def view(t):
        wide = torch.full((t.shape[0], t.shape[1] + 9), 7.0, dtype=dtype, device="cuda")
        v = wide[:, off:off + t.shape[1]]
        v.copy_(t)
        return wide, v

    _, xv = view(x)
    _, dyv = view(dy)
    wy, yv = view(torch.zeros(m, out, device="cuda"))
    wgx, gx = view(torch.zeros(m, d, device="cuda"))
    block = gsr().GatedFFN(wg, wu, wd)
    _, saved = block.forward(xv, y=yv, save=True)
    grads = block.new_grads(m)
    grads["x"] = gx
    block.backward(xv, saved, dyv, grads=grads)
    ref = o.ffn(x, wg, wu, wd, "silu", dy)
    o.check(yv, ref["y"], ffn_tol(dtype, 2, 144), "y")
    o.check(grads["w_down"], ref["w_down"], ffn_tol(dtype, 2, 144), "w_down")
    for name in ("x", "w_gate", "w_up"):
        o.check(grads[name], ref[name], ffn_tol(dtype, 4, 144), name)
    for wide, v in ((wy, out), (wgx, d)):
        rest = torch.cat([wide[:, :off], wide[:, off + v:]], dim=1)
        assert (rest == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_ffn_some_gradients_only_and_no_rows(dtype):
    x, wg, wu, wd, dy = ffn_inputs(40, 24, 56, 16, dtype, seed=5)
    block = gsr().GatedFFN(wg, wu, wd)
    _, saved = block.forward(x, save=True)
    full = block.backward(x, saved, dy)
    for names in (("x",), ("w_gate",), ("w_up",), ("w_down",), ("x", "w_up")):
        grads = {n: torch.full_like(full[n], 3.0) for n in names}
        block.backward(x, saved, dy, grads=grads)
        for n in names:
            assert torch.equal(grads[n], full[n]), n
    none = x[:0]
    y, saved = block.forward(none, save=True)
    assert y.shape == (0, 16)
    grads = block.backward(none, saved, dy[:0])
    for n in ("w_gate", "w_up", "w_down"):
        assert (grads[n] == 0).all(), n


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [5, 200])
def test_ffn_keeps_bad_rows_apart(dtype, rows):
    """A row with NaN or infinity spoils its own row of y and dx and nothing else; the workspace's old contents
    (NaN bit patterns) reach nothing."""
    x, wg, wu, wd, dy = ffn_inputs(rows, 50, 70, 30, dtype, seed=6)
    block = gsr().GatedFFN(wg, wu, wd)
    block._scratch(1 << 24, torch.cuda.current_stream()).fill_(255)
    y0, s0 = block.forward(x, save=True)
    block.workspace.fill_(255)
    g0 = block.backward(x, s0, dy)
    bad = x.clone()
    bad[2, 7] = float("nan")
    bad[4, 3] = float("inf")
    y1, s1 = block.forward(bad, save=True)
    g1 = block.backward(bad, s1, dy)
    keep = [r for r in range(rows) if r not in (2, 4)]
    assert torch.isfinite(y0).all() and torch.isfinite(g0["x"]).all()
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(g0["x"][keep], g1["x"][keep])
    assert torch.isnan(y1[2]).all() and not torch.isfinite(y1[4]).any()


def test_ffn_gradient_against_differences():
    """<grad, v> against the central difference of <y, dy> along v, float32.  Both sides of the difference carry
    float32 rounding: with |y| summing 60 x 20 products of size 1 the loss is known to about 1200^(1/2) 16 u = 3e-5,
    so a step of 1e-2 resolves 3e-3; the step's own third-order term is below 1e-4 of the derivative's scale, 35."""
    x, wg, wu, wd, dy = ffn_inputs(60, 30, 44, 20, torch.float32, seed=7)
    block = gsr().GatedFFN(wg, wu, wd, activation="gelu")
    _, saved = block.forward(x, save=True)
    grads = block.backward(x, saved, dy)
    eps = 1e-2
    for name, t in (("x", x), ("w_gate", wg), ("w_up", wu), ("w_down", wd)):
        v = randn(gen(8), *t.shape, scale=t.numel() ** -0.5)
        keep, side = t.clone(), []
        for sign in (1, -1):
            t.copy_(keep + sign * eps * v)
            side.append((block.forward(x).double() * dy.double()).sum().item())
        t.copy_(keep)
        diff = (side[0] - side[1]) / (2 * eps)
        assert abs(diff - (grads[name].double() * v.double()).sum().item()) <= 1e-2, name


def test_ffn_on_another_stream_and_far_rows():
    """Work queued on a side stream, and rows that lie more than 2^31 elements from the first."""
    dtype = torch.bfloat16
    x, wg, wu, wd, _ = ffn_inputs(1040, 64, 64, 32, dtype, seed=9)
    side = torch.cuda.Stream()
    wide = torch.empty((1040, 1 << 21), dtype=dtype, device="cuda")
    xv = wide[:, :64]
    xv.copy_(x)
    block = gsr().GatedFFN(wg, wu, wd)
    want = block.forward(x)
    side.wait_stream(torch.cuda.current_stream())
    y = block.forward(xv, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    o.check(y, o.ffn(x, wg, wu, wd, "silu"), ffn_tol(dtype, 2, 64), "y")


def test_ffn_refusals():
    m = gsr()
    w = torch.zeros(8, 4, device="cuda")
    wd = torch.zeros(3, 8, device="cuda")
    with pytest.raises(ValueError):
        m.GatedFFN(w, w, wd, activation="relu")
    with pytest.raises(ValueError):
        m.GatedFFN(w, w[:7], wd)
    with pytest.raises(ValueError):
        m.GatedFFN(w, w, wd.bfloat16())
    with pytest.raises(ValueError):
        m.GatedFFN(w.double(), w.double(), wd.double())
    with pytest.raises(ValueError):
        m.GatedFFN(w.cpu(), w.cpu(), wd.cpu())
    with pytest.raises(ValueError):
        m.GatedFFN(w, w, torch.zeros(8, 3, device="cuda").t())
    block = m.GatedFFN(w, w, wd)
    x = torch.zeros(5, 4, device="cuda")
    for bad in (x[:, :3], x.bfloat16(), x.cpu(), torch.zeros(4, 5, device="cuda").t(), x[0]):
        with pytest.raises((ValueError, IndexError)):
            block.forward(bad)
    with pytest.raises(ValueError):
        block.forward(x, y=torch.zeros(5, 4, device="cuda"))
    with pytest.raises(ValueError):
        block.backward(x, None, torch.zeros(5, 3, device="cuda"))


# ---- recurrence -----------------------------------------------------------------------------------------

def scan_case(rows, c, offsets, dtype, seed=0, gate_scale=1.5, gate_mean=1.0):
    g = gen(seed)
    z = (torch.randn(rows, c, generator=g, device="cuda") * gate_scale + gate_mean).to(dtype)
    n = len(offsets) - 1
    return (z, randn(g, rows, c, dtype=dtype), randn(g, n, c), randn(g, rows, c, dtype=dtype), randn(g, n, c),
            torch.tensor(offsets, dtype=torch.int64, device="cuda"))


def scan_check(z, x, h0, dy, dl, offsets, off_t, dtype, equal=False):
    c = x.shape[1]
    op = gsr().GatedScan(c, dtype)
    kw = dict(h0=h0, offsets=None if equal else off_t)
    y, hl = op.forward(z, x, **kw)
    y2, hl2, saved = op.forward(z, x, save=True, **kw)
    got = op.backward(z, x, saved, dy, dl, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(hl, hl2)
    cpu = [t.float().cpu().numpy() for t in (z, x, h0, dy, dl)]
    ref = o.scan(cpu[0], cpu[1], offsets, cpu[2], cpu[3], cpu[4])
    u32 = 32 * o.UNIT[torch.float32]
    u = o.UNIT[dtype] + u32 if dtype != torch.float32 else u32
    o.check(y, ref["y"], u, "y")
    o.check(hl, ref["h_last"], u32, "h_last")
    o.check(got["gate"], ref["gate"], u, "gate")
    o.check(got["x"], ref["x"], u, "x")
    o.check(got["h0"], ref["h0"], u32, "h0")
    return y, got


RAGGED = [[0, 1], [0, 127], [0, 128], [0, 129], [0, 0, 1, 1, 2], [0, 16, 16, 17, 128, 128, 128, 300],
          [0, 1, 2, 3, 4, 5, 6, 7, 400], [0, 1024, 1025, 2100], [0, 0, 0, 700, 700]]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("offsets", RAGGED, ids=lambda v: "-".join(map(str, v)))
def test_scan_ragged(offsets, dtype):
    scan_check(*scan_case(offsets[-1], 70, offsets, dtype)[:5], offsets,
               torch.tensor(offsets, dtype=torch.int64, device="cuda"), dtype)


@pytest.mark.parametrize("c", [1, 2, 3, 31, 32, 33, 64, 65, 66, 128, 129, 130, 258])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_scan_channels(c, dtype):
    offsets = [0, 100, 101, 333]
    scan_check(*scan_case(333, c, offsets, dtype, seed=1)[:5], offsets,
               torch.tensor(offsets, dtype=torch.int64, device="cuda"), dtype)


@pytest.mark.parametrize("length, n", [(1, 1), (1, 300), (3, 50), (128, 3), (64, 7), (96, 5), (20000, 1), (9001, 2)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scan_equal_lengths(length, n, dtype):
    offsets = [i * length for i in range(n + 1)]
    case = scan_case(length * n, 34, offsets, dtype, seed=2, gate_mean=3.0)
    y, got = scan_check(*case[:5], offsets, case[5], dtype, equal=True)
    y2, got2 = scan_check(*case[:5], offsets, case[5], dtype, equal=False)
    assert torch.equal(y, y2) and all(torch.equal(got[k], got2[k]) for k in got)


def test_scan_is_reproducible_over_many_chunks():
    offsets = [0, 150000]
    z, x, h0, dy, dl, off = scan_case(150000, 64, offsets, torch.float32, seed=3, gate_mean=6.0)
    op = gsr().GatedScan(64, torch.float32)
    first = None
    for _ in range(4):
        y, hl, saved = op.forward(z, x, h0=h0, offsets=off, save=True)
        g = op.backward(z, x, saved, dy, dl, h0=h0, offsets=off)
        now = [y, hl, g["gate"], g["x"], g["h0"]]
        if first is None:
            first = now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scan_extreme_gates(dtype):
    """Gates that keep or replace the state entirely, infinite ones included."""
    offsets = [0, 300]
    z, x, h0, dy, dl, off = scan_case(300, 40, offsets, dtype, seed=4)
    inf = float("inf")
    for i, v in enumerate((inf, -inf, 100.0, -100.0, 60000.0, -60000.0, 0.0)):
        z[i::7] = v
    scan_check(z, x, h0, dy, dl, offsets, off, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scan_keeps_sequences_apart(dtype):
    """NaN and infinities of one sequence stay in it, in both directions."""
    offsets = [0, 200, 200, 500, 501, 900]
    z, x, h0, dy, dl, off = scan_case(900, 48, offsets, dtype, seed=5)
    op = gsr().GatedScan(48, dtype)

    def run():
        y, hl, saved = op.forward(z, x, h0=h0, offsets=off, save=True)
        return (y, hl), op.backward(z, x, saved, dy, dl, h0=h0, offsets=off)

    (y0, l0), g0 = run()
    x[300] = float("nan")
    dy[350] = float("inf")
    z[400] = float("nan")
    h0[2], dl[2] = float("nan"), float("inf")
    (y1, l1), g1 = run()
    rows = torch.cat([torch.arange(200), torch.arange(500, 900)]).cuda()
    seqs = torch.tensor([0, 1, 3, 4]).cuda()
    for a, b_, i in ((y0, y1, rows), (l0, l1, seqs), (g0["gate"], g1["gate"], rows), (g0["x"], g1["x"], rows),
                     (g0["h0"], g1["h0"], seqs)):
        assert torch.equal(a[i], b_[i])
    assert torch.isnan(y1[499]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("off", [0, 1])
def test_scan_strides(dtype, off):
    """gate and x as halves of one projection, outputs in wider arrays, off the vector alignment."""
    offsets = [0, 150, 333]
    z, x, h0, dy, dl, offs = scan_case(333, 36, offsets, dtype, seed=6)
    op = gsr().GatedScan(36, dtype)
    y, hl, saved = op.forward(z, x, h0=h0, offsets=offs, save=True)
    g = op.backward(z, x, saved, dy, dl, h0=h0, offsets=offs)
    joint = torch.full((333, 80), 9.0, dtype=dtype, device="cuda")
    zv, xv = joint[:, off:off + 36], joint[:, 40 + off:76 + off]
    zv.copy_(z)
    xv.copy_(x)
    wide = torch.full((333, 120), 9.0, dtype=dtype, device="cuda")
    yv, gz, gx = (wide[:, k + off:k + off + 36] for k in (0, 40, 80))
    y2, hl2, saved2 = op.forward(zv, xv, h0=h0, offsets=offs, y=yv, save=True)
    op.backward(zv, xv, saved2, dy, dl, h0=h0, offsets=offs, grads={"gate": gz, "x": gx})
    for a, b_ in ((y, yv), (hl, hl2), (g["gate"], gz), (g["x"], gx)):
        assert torch.equal(a, b_)
    assert (wide[:, 36 + off:40] == 9.0).all() and (wide[:, 116 + off:] == 9.0).all()


def test_scan_optional_arrays_and_steps():
    """No h0, no dh_last; the state carried over single steps in place equals one long pass."""
    dtype, c, n, steps = torch.bfloat16, 96, 50, 12
    g = gen(7)
    z, x = randn(g, n, steps, c, dtype=dtype), randn(g, n, steps, c, dtype=dtype)
    op = gsr().GatedScan(c, dtype)
    off = torch.arange(n + 1, device="cuda") * steps
    y, hl = op.forward(z.view(-1, c), x.view(-1, c), offsets=off)
    h = torch.zeros(n, c, device="cuda")
    for t in range(steps):
        yt, _ = op.forward(z[:, t].contiguous(), x[:, t].contiguous(), h0=h, h_last=h)
        assert torch.equal(yt, y.view(n, steps, c)[:, t])
    assert torch.equal(h, hl)
    y1, _, saved = op.forward(z.view(-1, c), x.view(-1, c), offsets=off, save=True)
    got = op.backward(z.view(-1, c), x.view(-1, c), saved, x.view(-1, c), offsets=off)
    zero = torch.zeros(n, c, device="cuda")
    want = op.backward(z.view(-1, c), x.view(-1, c), saved, x.view(-1, c), zero, h0=zero, offsets=off)
    assert all(torch.equal(got[k], want[k]) for k in got)
    none, h_last = op.forward(z.view(-1, c)[:0], x.view(-1, c)[:0], h0=h, offsets=torch.zeros(n + 1, dtype=torch.int64,
                                                                                           device="cuda"))
    assert none.shape == (0, c) and torch.equal(h_last, h)


def test_scan_far_rows():
    """Rows more than 2^31 elements apart."""
    dtype, rows, c = torch.bfloat16, 1100, 64
    z, x, h0, _, _, off = scan_case(rows, c, [0, rows], dtype, seed=8)
    op = gsr().GatedScan(c, dtype)
    want, last = op.forward(z, x, h0=h0, offsets=off)
    wide = torch.empty((rows, 1 << 21), dtype=dtype, device="cuda")
    zv, xv, yv = (wide[:, k:k + c] for k in (0, 64, 128))
    zv.copy_(z)
    xv.copy_(x)
    _, last2 = op.forward(zv, xv, h0=h0, offsets=off, y=yv)
    assert torch.equal(yv, want) and torch.equal(last, last2)


def test_scan_odd_offsets_stay_in_range():
    """Offsets that do not start at 0, do not end at the last row or lie outside the rows: no access out of range
    (the arrays around them keep their values)."""
    c, rows = 33, 300
    z, x, _, dy, _, _ = scan_case(rows, c, [0, rows], torch.float32, seed=9)
    op = gsr().GatedScan(c, torch.float32)
    for offs in ([5, 100, 250], [0, 10, 100000], [-40, 7, 299], [100, 50, 10, 300], [10 ** 12, 5, -10 ** 12, 3]):
        off = torch.tensor(offs, dtype=torch.int64, device="cuda")
        n = len(offs) - 1
        guard = torch.full((3, n + 2, c), 4.0, device="cuda")
        guard[0, 1:-1] = 0.0
        y, _, saved = op.forward(z, x, h0=guard[0, 1:-1], offsets=off, h_last=guard[1, 1:-1], save=True)
        op.backward(z, x, saved, dy, None, h0=guard[0, 1:-1], offsets=off, grads={"h0": guard[2, 1:-1]})
        torch.cuda.synchronize()
        assert (guard[:, 0] == 4.0).all() and (guard[:, -1] == 4.0).all()


def test_scan_refusals():
    op = gsr().GatedScan(8, torch.float32)
    z = torch.zeros(12, 8, device="cuda")
    with pytest.raises(ValueError):
        op.forward(z, z[:, :7])
    with pytest.raises(ValueError):
        op.forward(z, z[:11])
    with pytest.raises(ValueError):
        op.forward(z.half(), z.half())
    with pytest.raises(ValueError):
        op.forward(z, z, h0=torch.zeros(2, 8, device="cuda").half())
    with pytest.raises(ValueError):
        op.forward(z, z, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(gsr().GsrError):
        op.forward(z, z, h0=torch.zeros(5, 8, device="cuda"))  # 12 rows are not 5 equal sequences
    with pytest.raises(ValueError):
        op.backward(z, z, None, z)
    with pytest.raises(ValueError):
        gsr().GatedScan(8, torch.float64)


# ---- orthogonalisation ----------------------------------------------------------------------------------

def ortho_tol(out):
    return 15 * 2.0 ** -12 + 2.0 ** -9 if out == torch.bfloat16 else 30 * 2.0 ** -22


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 40), (2, 40, 1), (3, 8, 8), (2, 33, 70), (2, 70, 33),
                                   (1, 130, 129), (4, 64, 200), (3, 200, 64), (1, 257, 300), (2, 300, 511)], ids=str)
@pytest.mark.parametrize("din, dout", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.float32), (torch.bfloat16, torch.float32)], ids=str)
def test_ortho(shape, din, dout):
    g = randn(gen(sum(shape)), *shape, scale=0.02, dtype=din)
    out = gsr().Orthogonalizer(*shape, din, dout).run(g)
    for got, m in zip(out, g):
        o.check(got, o.newton_schulz(m, 5, NS), ortho_tol(dout), "out")


@pytest.mark.parametrize("shape", [(1, 2100, 2200), (1, 2200, 2048), (8, 1000, 1100)], ids=str)
def test_ortho_large(shape):
    g = randn(gen(1), *shape, dtype=torch.float32)
    for dout in (torch.bfloat16, torch.float32):
        out = gsr().Orthogonalizer(*shape, torch.float32, dout).run(g)
        o.check(out[-1], o.newton_schulz(g[-1], 5, NS), ortho_tol(dout), "out")


def test_ortho_orthogonal_rows_and_scale():
    """Exactly orthogonal rows keep their directions: each row ends with the polynomial's value of 1 / sqrt(rows),
    whatever the scale of the input (checked from 2^-60 to 2^60)."""
    rows, cols = 4, 64
    s = rows ** -0.5
    for _ in range(5):
        s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
    for scale in (2.0 ** -60, 1.0, 2.0 ** 60):
        g = torch.zeros(1, rows, cols, device="cuda")
        for r in range(rows):
            g[0, r, r * 7] = scale
        out = gsr().Orthogonalizer(1, rows, cols, torch.float32, torch.float32, eps=1e-30).run(g)
        want = torch.zeros(rows, cols, dtype=torch.float64)
        for r in range(rows):
            want[r, r * 7] = s
        o.check(out[0], want, ortho_tol(torch.float32), "out")


def test_ortho_zero_and_bad_matrices():
    """A zero matrix gives zeros; NaN and infinity spoil their own matrix only."""
    g = randn(gen(2), 4, 48, 80)
    op = gsr().Orthogonalizer(4, 48, 80, torch.float32, torch.bfloat16)
    want = op.run(g)
    g[1] = 0
    g[2, 5, 5] = float("nan")
    g[3, 1, 2] = float("inf")
    got = op.run(g)
    assert torch.equal(got[0], want[0]) and (got[1] == 0).all()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).any()


def test_ortho_repeats_and_refuses():
    m = gsr()
    g = randn(gen(3), 2, 100, 60)
    op = m.Orthogonalizer(2, 100, 60, torch.float32, torch.bfloat16, steps=3, coefficients=(1.5, -0.5, 0.0))
    first = op.run(g)
    op.workspace.fill_(255)
    assert torch.equal(first, op.run(g))
    o.check(first[1], o.newton_schulz(g[1], 3, (1.5, -0.5, 0.0)), ortho_tol(torch.bfloat16), "out")
    one = m.Orthogonalizer(1, 100, 60, torch.float32, torch.bfloat16, steps=3, coefficients=(1.5, -0.5, 0.0))
    assert torch.equal(one.run(g[0]), first[0])
    for bad in (g[0], g.half(), g.cpu(), g.transpose(1, 2)):
        with pytest.raises(ValueError):
            op.run(bad)
    with pytest.raises(ValueError):
        op.run(g, out=torch.zeros(2, 100, 60, device="cuda"))
    with pytest.raises(ValueError):
        m.Orthogonalizer(1, 4, 4, torch.float16)
    with pytest.raises(m.GsrError):
        m.Orthogonalizer(1, 4, 4, torch.float32, steps=0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(130, 60, 76, 20), (70, 12, 100, 36)], ids=str)
def test_ffn_ends_of_arrays(shape, dtype):
    """Row lengths of 4 modulo 8 with arrays that end where NaN begins."""
    m, d, f, out = shape
    tensors = ffn_inputs(m, d, f, out, dtype, seed=43)

    def end(t):
        room = torch.full((t.numel() + 64,), float("nan"), dtype=dtype, device="cuda")
        room[:t.numel()] = t.flatten()
        return room[:t.numel()].view(t.shape)

    x, wg, wu, wd, dy = (end(t) for t in tensors)
    block = gsr().GatedFFN(wg, wu, wd)
    y, saved = block.forward(x, save=True)
    got = block.backward(x, saved, dy)
    ref = o.ffn(*tensors[:4], "silu", tensors[4])
    k = max(m, 2 * f, d, out)
    o.check(y, ref["y"], ffn_tol(dtype, 2, k), "y")
    o.check(got["w_down"], ref["w_down"], ffn_tol(dtype, 2, k), "w_down")
    for name in ("x", "w_gate", "w_up"):
        o.check(got[name], ref[name], ffn_tol(dtype, 4, k), name)


def test_all_in_a_graph():
    """Training form of block and recurrence, single-step forms and both orthogonalisations, captured once and replayed
    with new inputs and other work in between: every replay equals the eager calls."""
    m, d, f, out, n = 200, 40, 72, 48, 5
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, torch.bfloat16, seed=40)
    g = gen(41)
    block = gsr().GatedFFN(wg, wu, wd)
    scan = gsr().GatedScan(24, torch.bfloat16)
    small, large = gsr().Orthogonalizer(2, 30, 50, torch.float32), gsr().Orthogonalizer(1, 150, 180, torch.bfloat16)
    h0 = randn(g, n, 24)
    offsets = torch.tensor([0, 7, 7, 90, 91, m], device="cuda")
    m1, m2 = randn(g, 2, 30, 50), randn(g, 150, 180, dtype=torch.bfloat16)

    def run():
        y, saved = block.forward(x, save=True)
        grads = block.backward(x, saved, dy)
        z, v = y[:, :24], y[:, 24:]
        s, last, kept = scan.forward(z, v, h0=h0, offsets=offsets, save=True)
        sg = scan.backward(z, v, kept, s, dh_last=last, h0=h0, offsets=offsets)
        one = block.forward(x[:1])
        step, state = scan.forward(z[:n], v[:n], h0=h0)
        return [y, s, last, one, step, state, small.run(m1), large.run(m2), *grads.values(), *sg.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        x.copy_(randn(g, m, d, dtype=torch.bfloat16))
        h0.copy_(randn(g, n, 24))
        m1.copy_(randn(g, 2, 30, 50))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = run()
        torch.cuda.synchronize()
        for k, (a, w) in enumerate(zip(got, want)):
            assert torch.equal(a, w), (i, k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("c, offsets", [
    (70, [0, 2]), (70, [0, 300]), (40, [0, 7, 9, 15, 17, 400]), (70, [0, 63, 65, 65, 129, 1500, 1501, 2600]),
    (70, [0, 0, 5, 700, 700]), (64, [0, 150000]), (130, [0, 40000, 40001, 90000])], ids=lambda v: str(v).replace(" ", ""))
def test_scan_in_place(c, offsets, dtype):
    """h_last in h0's memory and dh0 in dh_last's, for sequences within a span, over spans, chunks and many chunks, with
    offsets and (where the lengths allow) without: y, states, what is saved and the gradients are what separate arrays
    give."""
    z, x, h0, dy, dl, off = scan_case(offsets[-1], c, offsets, dtype, seed=11, gate_mean=4.0)
    op = gsr().GatedScan(c, dtype)
    lengths = {b_ - a for a, b_ in zip(offsets, offsets[1:])}
    for kw in [dict(offsets=off)] + ([dict()] if len(lengths) == 1 else []):
        y, hl, saved = op.forward(z, x, h0=h0, save=True, **kw)
        want = op.backward(z, x, saved, dy, dl, h0=h0, **kw)
        state = h0.clone()
        y2, hl2, saved2 = op.forward(z, x, h0=state, h_last=state, save=True, **kw)
        assert hl2 is state
        assert torch.equal(y2, y) and torch.equal(state, hl)
        n = (offsets[-1] + 7) // 8 * c * 4
        assert torch.equal(saved2[:n], saved[:n])
        end = dl.clone()
        got = {"gate": torch.empty_like(z), "x": torch.empty_like(x), "h0": end}
        op.backward(z, x, saved, dy, end, h0=h0, grads=got, **kw)
        assert all(torch.equal(got[k], want[k]) for k in want)
        start = h0.clone()
        op.backward(z, x, saved, dy, dl, h0=start, grads={"h0": start}, **kw)
        assert torch.equal(start, want["h0"])


@pytest.mark.parametrize("shape", [(1, 1, 40), (2, 33, 70), (1, 70, 33), (2, 128, 192), (1, 1, 2100), (1, 300, 511)],
                         ids=str)
@pytest.mark.parametrize("dout", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("coef, steps", [((3.0, -0.1, 0.0), 2), ((8.2872, -23.5959, 17.3004), 1), ((15.0, 0.0, 0.0), 2)],
                         ids=str)
def test_ortho_coefficients_near_the_limit(coef, steps, dout, shape):
    """Coefficients that take P, Q or X past what the default scales hold, in the one-workgroup and the tiled form.
    Error of a step, first order, u = 2^-11 (bfloat16 result) or 2^-20 (pairs): what came in times |p'(s)|, and every
    factor of every term rounded once -- X in a s, X X X P and twice Q in b s^3, five X, two P and twice Q in c s^5 --
    and the result; summed over the singular values, plus the result's own rounding."""
    g = randn(gen(sum(shape)), *shape, dtype=torch.float32)
    out = gsr().Orthogonalizer(*shape, torch.float32, dout, steps=steps, coefficients=coef).run(g)
    a, b_, c = coef
    u = 2.0 ** -11 if dout == torch.bfloat16 else 2.0 ** -20
    for got, m in zip(out, g):
        s = torch.linalg.svdvals(m.double().cpu())
        s = s / s.norm()
        e = u * s
        for _ in range(steps):
            slope = (a + 3 * b_ * s ** 2 + 5 * c * s ** 4).abs()
            own = abs(a) * s + 6 * abs(b_) * s ** 3 + 9 * abs(c) * s ** 5
            s = a * s + b_ * s ** 3 + c * s ** 5
            e = slope * e + u * (own + s.abs())
        tol = (e.norm() / s.norm()).item() + (o.UNIT[dout] if dout == torch.bfloat16 else 0.0)
        o.check(got, o.newton_schulz(m, steps, coef), tol, "out")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [50, 800])
def test_gelu_tail(rows, dtype):
    """One hidden unit with u = 1 and dy = 1, element by element into the far tail: y and du are g Phi(g), dg is
    Phi(g) + g phi(g) (relative to its two terms), each rounded to the type once.  Before that, float32 loses g^2 u to
    the exponential's argument and a dozen u to the rest; for the 16-bit types Phi is good to 1e-5.  Results below the
    type's normal numbers are good to half its least one."""
    g = torch.linspace(-12, 8, rows, device="cuda").to(dtype)
    one = torch.ones(rows, 1, device="cuda", dtype=dtype)
    x = torch.cat([g[:, None], one], dim=1)
    wg, wu = (torch.tensor([v], device="cuda", dtype=dtype) for v in ([1.0, 0.0], [0.0, 1.0]))
    block = gsr().GatedFFN(wg, wu, one[:1], activation="gelu")
    y, saved = block.forward(x, save=True)
    dx = block.backward(x, saved, one)["x"].double()
    g = g.double()
    cdf, gpdf = torch.special.erfc(-g / math.sqrt(2)) / 2, g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    rel = o.UNIT[dtype] + (1e-5 if dtype != torch.float32 else (12 + 1.5 * g * g) * o.UNIT[dtype])
    least = torch.finfo(dtype).smallest_normal * o.UNIT[dtype]
    for got, want, scale in ((y[:, 0].double(), g * cdf, g * cdf), (dx[:, 1], g * cdf, g * cdf),
                             (dx[:, 0], cdf + gpdf, cdf + gpdf.abs())):
        worst = (got - want).abs() / (rel * scale.abs() + least)
        assert worst.max() <= 1.0, (worst.max(), g[worst.argmax()])


def test_larger_call_after_a_capture():
    """The graph's scratch memory stays its own: a replay after a larger eager call gives the captured results and
    writes into nothing that was allocated meanwhile."""
    x, wg, wu, wd, dy = ffn_inputs(100, 40, 72, 48, torch.bfloat16, seed=50)
    block = gsr().GatedFFN(wg, wu, wd)

    def run():
        y, saved = block.forward(x, save=True)
        return [y, *block.backward(x, saved, dy).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    small = block.workspace.numel()
    big, *_ = ffn_inputs(5000, 40, 72, 48, torch.bfloat16, seed=51)
    want_big = block.forward(big)
    assert block.workspace.numel() > small
    filled = [torch.full((small,), 77, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for i in range(3):
        x.copy_(randn(gen(52 + i), 100, 40, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, w) for a, w in zip(got, run())), i
        assert all((f == 77).all() for f in filled) and torch.equal(block.forward(big), want_big)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [5, 200])
def test_float16_gates_beyond_the_range(rows, act):
    """Row 0 drives half of the gates to 120000 and closes the others at -120000, row 1 drives u to 120000: beyond
    float16's 65504 while h, y and every gradient are within it.  Tolerances as everywhere."""
    d, f, out = 24, 16, 8
    x, wg, wu, wd, dy = ffn_inputs(rows, d, f, out, torch.float16, seed=60)
    x[:2], x[:, :2] = 0, 0
    x[0, 0] = x[1, 1] = 300
    wg[0::2, 0], wg[1::2, 0], wu[:, 0] = 400, -400, 0.25 / 300
    wg[:, 1], wu[:, 1] = -1 / 300, 400
    dy[:2] *= 2.0 ** -12
    block = gsr().GatedFFN(wg, wu, wd, activation=act)
    y, saved = block.forward(x, save=True)
    got = block.backward(x, saved, dy)
    ref = o.ffn(x, wg, wu, wd, act, dy)
    for k in (slice(0, 1), slice(1, 2), slice(2, None)):
        o.check(y[k], ref["y"][k], ffn_tol(torch.float16, 2, 0), "y")
        o.check(got["x"][k], ref["x"][k], ffn_tol(torch.float16, 4, 0), "x")
    o.check(got["w_down"], ref["w_down"], ffn_tol(torch.float16, 2, 0), "w_down")
    for name in ("w_gate", "w_up"):
        o.check(got[name], ref[name], ffn_tol(torch.float16, 4, 0), name)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(3, 40, 1500, 2050), (20, 72, 2048, 1100), (50, 33, 2056, 1999)], ids=str)
def test_ffn_few_rows_wide(shape, dtype):
    """Few rows on both sides of 2048 columns, where the workgroups' width changes."""
    x, wg, wu, wd, _ = ffn_inputs(*shape, dtype, seed=70)
    y = gsr().GatedFFN(wg, wu, wd).forward(x)
    o.check(y, o.ffn(x, wg, wu, wd, "silu"), ffn_tol(dtype, 2, max(shape)), "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", [(40, 192, 640, 256), (700, 320, 1000, 200)], ids=str)
def test_ffn_gradients_carry_two_roundings(shape, act, dtype):
    """Rounding to nearest is off by 0.4247 u in the mean (root mean square over a mantissa spread evenly in its
    logarithm).  Every result carries two independent ones, the operand's and its own: sqrt(2) of that in its L2 error,
    and 6 % for everything else (four, with g and u kept in the type, would be up to 2)."""
    x, wg, wu, wd, dy = ffn_inputs(*shape, dtype, seed=80)
    block = gsr().GatedFFN(wg, wu, wd, activation=act)
    y, saved = block.forward(x, save=True)
    got = dict(block.backward(x, saved, dy), y=y)
    for k, ref in o.ffn(x, wg, wu, wd, act, dy).items():
        err = ((got[k].double() - ref).norm() / ref.norm()).item()
        assert err <= 1.5 * 0.4247 * o.UNIT[dtype], (k, err / (0.4247 * o.UNIT[dtype]))


@pytest.mark.parametrize("shape", [(12, 40, 77), (12, 108, 39), (12, 128, 512), (2, 200, 300)], ids=str)
def test_ortho_small_operand_error(shape):
    """float16 operands (2^-12 a rounding) may add as much to a bfloat16 result's error as its own rounding (0.4247 2^-8
    in the mean): sqrt(2) of that in all, and 3 % for the batch's spread.  The default coefficients' terms nearly cancel
    on singular values near 1, where Q holding them apart would cost 1.56."""
    g = randn(gen(90), *shape)
    out = gsr().Orthogonalizer(*shape, torch.float32, torch.bfloat16).run(g)
    ref = torch.stack([o.newton_schulz(m, 5, NS) for m in g])
    err = ((out.double() - ref).norm() / ref.norm()).item()
    assert err <= 1.45 * 0.4247 * 2.0 ** -8, err / (0.4247 * 2.0 ** -8)


@pytest.mark.parametrize("shape", [(200, 64, 6000, 48), (1500, 48, 3100, 64)], ids=str)
def test_ffn_float32_long_sums(shape):
    """A rounding is off by 0.4247 u in the mean.  A sum of K float32 terms in chains of 256 carries sqrt(128 + K / 512)
    of them (one chain: sqrt(K / 2), 55 of them for K = 6000, 77 for dx's 12000), the sums in front of it of up to 64
    terms and two more operands sqrt(4 * 64); half as much again for the activations."""
    m, d, f, out = shape
    x, wg, wu, wd, dy = ffn_inputs(*shape, torch.float32, seed=91)
    block = gsr().GatedFFN(wg, wu, wd)
    y, saved = block.forward(x, save=True)
    dx = block.backward(x, saved, dy)["x"]
    ref = o.ffn(x, wg, wu, wd, "silu", dy)
    for got, want, k in ((y, ref["y"], f), (dx, ref["x"], 2 * f)):
        err = ((got.double() - want).norm() / want.norm()).item()
        tol = 1.5 * 0.4247 * o.UNIT[torch.float32] * math.sqrt(128 + k / 512 + 4 * 64)
        assert err <= tol, (err, tol)


def test_ffn_a_billion_rows():
    """More tiles of 64 rows than a launch has room for: larger tiles take them.  One input, hidden unit and output each,
    y = silu(x) x to two roundings."""
    rows = (1 << 30) + 3
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 1 << 27):
        x[i:i + (1 << 27)].normal_(generator=gen(i >> 27))
    one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    y = gsr().GatedFFN(one, one, one).forward(x)
    for i in range(0, rows, 1 << 27):
        v = x[i:i + (1 << 27)].float()
        want = v * torch.sigmoid(v) * v
        assert ((y[i:i + (1 << 27)].float() - want).abs() <= 2.1 * o.UNIT[torch.bfloat16] * want + 1e-37).all(), i


def test_ffn_float32_few_rows_of_a_large_block():
    """Few rows whose backward pass runs on split operands: the forward pass keeps h in both forms."""
    m, d, f, out = 64, 2048, 16384, 4608
    x, wg, wu, wd, dy = ffn_inputs(m, d, f, out, torch.float32, seed=92)
    block = gsr().GatedFFN(wg, wu, wd)
    y, saved = block.forward(x, save=True)
    assert torch.equal(block.forward(x), y)
    got = block.backward(x, saved, dy)
    ref = o.ffn(x, wg, wu, wd, "silu", dy)
    tol = ffn_tol(torch.float32, 0, 2 * f)
    o.check(y, ref["y"], tol, "y")
    for name in ("x", "w_gate", "w_up", "w_down"):
        o.check(got[name], ref[name], tol, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("mean", [6.0, 8.0, 10.0, 12.0])
def test_scan_long_memory(mean, dtype):
    """Gates that keep the state for 400 to 160,000 rows.  The tolerances of the recurrence, which do not grow with the
    memory: a itself, rounded next to 1, would leave the state 2^-25 / (1 - a) off, 1.4e-4 for gates of 10."""
    rows, c = 40000, 6
    g = gen(93)
    z = (torch.randn(rows, c, generator=g, device="cuda") * 0.1 + mean).to(dtype)
    x, dy = ((torch.randn(rows, c, generator=g, device="cuda") + 1).to(dtype) for _ in range(2))
    offsets = [0, 39000, rows]
    h0, dl = randn(g, 2, c), randn(g, 2, c)
    scan_check(z, x, h0, dy, dl, offsets, torch.tensor(offsets, device="cuda"), dtype)
