"""Linear attention on the GPU against its definition in float64.

Tolerances (relative L2; per element see updater_oracle.check), u = unit roundoff of the type, V = 2^-24, T = the longest
sequence (at least the 128 products of a row with the state):
- y: one rounding to the type; float32: products to 24 bits, sums of T terms in chains of 16, the decays' exponentials: 32 V
  and 2 sqrt(T) V.  16-bit: state and scores as operands of 16 bits in products that leave out 2^-16: 2^-15 more.
- last, gradient of state, in float32 for every type: 32 V + 2 sqrt(T) V.
- gradients of q, k, v: u, and 64 V + 4 sqrt(T) V, two passes in a row.
- gradient of the gate: sums of products of two results, differences within a chunk and from chunk to chunk of one span (at
  most 32 + 64 of them): 128 V + 8 sqrt(T) V, and its type's rounding.
"""
import pytest
import torch

import attention_oracle as ao
import updater_oracle as o

pytestmark = pytest.mark.gpu
V = ao.V
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def inputs(rows, n_seq, H, K, dk, dv, dtype, gate="rows", seed=0, gate_dtype=torch.float32, bias=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, scale=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    x = {"q": r(rows, H, dk), "k": r(rows, K, dk, scale=dk ** -0.5), "v": r(rows, K, dv),
         "gate": (r(*((rows, K) if gate == "rows" else (K,)), scale=1.5, dtype=torch.float32) + bias).to(gate_dtype),
         "state": r(n_seq, K, dk, dv, dtype=torch.float32)}
    return x, r(rows, H, dv), r(n_seq, K, dk, dv, scale=0.3, dtype=torch.float32)


def tols(dtype, T, gate_dtype=torch.float32):
    T = max(T, 128)
    u = 0 if dtype == torch.float32 else o.UNIT[dtype]
    y = u + (2.0 ** -15 if u else 0) + (32 + 2 * ao.root(T)) * V
    g = u + (64 + 4 * ao.root(T)) * V
    gu = 0 if gate_dtype == torch.float32 else o.UNIT[gate_dtype]
    return {"y": y, "last": (32 + 2 * ao.root(T)) * V, "q": g, "k": g, "v": g, "state": (64 + 4 * ao.root(T)) * V,
            "gate": gu + (128 + 8 * ao.root(T)) * V}


def check_all(H, K, dk, dv, dtype, lengths, ragged, gate="rows", gate_dtype=torch.float32, seed=0, bias=3.0, tail=0):
    rows, n_seq = sum(lengths), len(lengths)
    x, dy, d_last = inputs(rows + tail, n_seq, H, K, dk, dv, dtype, gate, seed, gate_dtype, bias)
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    offsets = torch.tensor(off, device="cuda") if ragged else None
    att = gsr().LinearAttention(H, dk, dv, dtype, kv_heads=K)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last = att.forward(*args, state=x["state"], offsets=offsets)
    y2, last2, saved = att.forward(*args, state=x["state"], offsets=offsets, save=True)
    assert torch.equal(y[:rows], y2[:rows]) and torch.equal(last, last2)
    got = att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=offsets)
    cut = {n: x[n][:rows] if n in ("q", "k", "v") or (n == "gate" and gate == "rows") else x[n] for n in x}
    ref = ao.attention(cut["q"], cut["k"], cut["v"], cut["gate"], off, x["state"], dk ** -0.5, dy[:rows], d_last)
    tol = tols(dtype, max(lengths, default=0), gate_dtype)
    got = {**{n: t[:rows] if n in ("q", "k", "v") or (n == "gate" and gate == "rows") else t for n, t in got.items()},
           "y": y[:rows], "last": last}
    for n in ("y", "last", "v", "k", "q", "state", "gate"):
        assert got[n].dtype == (x[n].dtype if n in x else dtype if n == "y" else torch.float32)
        o.check(got[n], ref[n], tol[n], n)
    return att, args, x, dy, d_last, offsets, saved, got


HEADS = [(1, 1, 1, 1), (1, 1, 64, 64), (2, 2, 8, 16), (4, 2, 64, 64), (3, 1, 57, 72), (2, 2, 128, 128), (4, 1, 128, 40),
         (6, 2, 33, 128), (8, 2, 100, 101)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_heads_and_widths(heads, dtype):
    check_all(*heads, dtype, [70], False)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 160, 257, 700])
def test_lengths(length, dtype):
    """One sequence: single rows, chunks and spans (128 rows here) that end in and between tiles."""
    check_all(2, 1, 64, 72, dtype, [length], False, seed=length)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("gate", ["rows", "heads"])
def test_ragged(gate, dtype):
    lengths = [5, 0, 0, 130, 1, 300, 64, 0, 129, 31, 33, 128, 256, 2, 0]
    check_all(4, 2, 57, 40, dtype, lengths, True, gate=gate, seed=2)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n_seq, length", [(5, 16), (3, 150), (40, 1), (7, 3)])
def test_equal_lengths(n_seq, length, dtype):
    check_all(4, 2, 64, 64, dtype, [length] * n_seq, False, gate="heads", seed=3)


@pytest.mark.parametrize("n_seq, ragged", [(200, True), (90, True)])
def test_many_sequences(n_seq, ragged):
    """More sequences than one probe of the search looks at, empty ones among them."""
    g = torch.Generator().manual_seed(n_seq)
    lengths = [int(v) if v < 25 else int(v) * 9 for v in torch.randint(0, 30, (n_seq,), generator=g)]
    check_all(2, 2, 16, 24, torch.float32, lengths, ragged, seed=4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_long_spans(dtype):
    """Enough rows for spans longer than the shortest ones: 16 key heads."""
    check_all(16, 16, 16, 16, dtype, [9000 - 37, 37, 3600], True, seed=5)


def test_rows_behind_the_last_sequence_are_left():
    x, dy, d_last = inputs(300, 2, 2, 2, 64, 64, torch.bfloat16, seed=6)
    offsets = torch.tensor([0, 130, 200], device="cuda")
    att = gsr().LinearAttention(2, 64, 64, torch.bfloat16)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y = torch.full((300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, saved = att.forward(*args, state=x["state"], offsets=offsets, y=y, save=True)
    grads = {n: torch.full_like(x[n], 7.0) for n in x}
    att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=offsets, grads=grads)
    for t in (y, grads["q"], grads["k"], grads["v"], grads["gate"]):
        assert (t[200:] == 7).all() and not (t[:200] == 7).all()
    check_all(2, 2, 64, 64, torch.bfloat16, [130, 70], True, seed=6, tail=100)


@pytest.mark.parametrize("gate_dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("bias", [-8.0, 0.0, 12.0])
def test_gates(bias, gate_dtype):
    """Heads that forget at once, and heads that keep nearly everything."""
    check_all(2, 2, 64, 64, torch.bfloat16, [400], False, gate_dtype=gate_dtype, bias=bias, seed=7)


def test_gates_that_reset_and_keep():
    """Infinite gates: a reset shuts out what was before it exactly, and a gate of infinity keeps everything."""
    x, dy, d_last = inputs(300, 1, 2, 2, 32, 32, torch.float32, seed=8)
    x["gate"][150] = -float("inf")
    x["gate"][40:60] = float("inf")
    x["gate"][200] = -200.0
    att = gsr().LinearAttention(2, 32, 32, torch.float32)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last, saved = att.forward(*args, state=x["state"], save=True)
    got = att.backward(*args, saved, dy, d_last=d_last, state=x["state"])
    ry, rl = ao.recurrence(*args, [0, 300], x["state"], 32 ** -0.5)
    tol = tols(torch.float32, 300)
    o.check(y, ry, tol["y"], "y")
    o.check(last, rl, tol["last"], "last")
    early = dy.clone()  # nothing from the reset on reaches the first state
    early[150:] = 0
    only = {"state": torch.empty_like(x["state"])}
    att.backward(*args, saved, early, state=x["state"], grads=only)
    assert torch.equal(only["state"], got["state"])
    assert (got["gate"][40:60] == 0).all() and (got["gate"][150] == 0).all()
    cut = {n: x[n][200:] if n != "state" else torch.zeros_like(x[n]) for n in x}  # after the last reset, by itself
    cut["gate"] = cut["gate"].clone()
    ref = ao.attention(cut["q"], cut["k"], cut["v"], cut["gate"], [0, 100], cut["state"], 32 ** -0.5, dy[200:], d_last)
    for n in ("q", "k", "v"):
        o.check(got[n][200:], ref[n], tol[n], n)
    o.check(got["gate"][201:], ref["gate"][1:], tol["gate"], "gate")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_and_alignment(dtype):
    """Slices of one projection, heads before rows, rows that start at odd elements: the same bits as contiguous ones."""
    T, H, K, dk, dv = 200, 4, 2, 40, 24
    x, dy, d_last = inputs(T, 1, H, K, dk, dv, dtype, seed=9)
    att = gsr().LinearAttention(H, dk, dv, dtype, kv_heads=K)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last, saved = att.forward(*args, state=x["state"], save=True)
    got = att.backward(*args, saved, dy, d_last=d_last, state=x["state"])
    wide = torch.zeros(T, 1 + H * dk + K * dk + K * dv + 3, dtype=dtype, device="cuda")
    q = wide[:, 1:1 + H * dk].view(T, H, dk)
    k = wide[:, 1 + H * dk:1 + (H + K) * dk].view(T, K, dk)
    v = wide[:, 1 + (H + K) * dk:1 + (H + K) * dk + K * dv].view(T, K, dv)
    for a, c in ((q, args[0]), (k, args[1]), (v, args[2])):
        a.copy_(c)
    gate = torch.zeros(T, K + 5, device="cuda")[:, 2:2 + K]
    gate.copy_(args[3])
    yt = torch.zeros(H, T, dv, dtype=dtype, device="cuda").transpose(0, 1)
    dyt = dy.transpose(0, 1).contiguous().transpose(0, 1)
    _, last2, saved2 = att.forward(q, k, v, gate, state=x["state"], y=yt, save=True)
    grads = torch.full_like(wide, 7.0)
    gg = torch.zeros(T, K + 1, device="cuda")[:, 1:]
    out = {"q": grads[:, 1:1 + H * dk].view(T, H, dk), "k": grads[:, 1 + H * dk:1 + (H + K) * dk].view(T, K, dk),
           "v": grads[:, 1 + (H + K) * dk:1 + (H + K) * dk + K * dv].view(T, K, dv), "gate": gg}
    att.backward(q, k, v, gate, saved2, dyt, d_last=d_last, state=x["state"], grads=out)
    assert torch.equal(yt, y) and torch.equal(last2, last)
    for n in out:
        assert torch.equal(out[n], got[n]), n
    assert (grads[:, 0] == 7).all() and (grads[:, -3:] == 7).all()


def test_heads_that_share_memory():
    """One key and value head given as several by a stride of zero."""
    x, _, _ = inputs(90, 1, 4, 1, 32, 32, torch.bfloat16, gate="heads", seed=10)
    one = gsr().LinearAttention(4, 32, 32, torch.bfloat16, kv_heads=1)
    y, last = one.forward(x["q"], x["k"], x["v"], x["gate"], state=x["state"])
    four = gsr().LinearAttention(4, 32, 32, torch.bfloat16)
    y2, last2 = four.forward(x["q"], x["k"].expand(90, 4, 32), x["v"].expand(90, 4, 32), x["gate"].expand(4).contiguous(),
                             state=x["state"].expand(1, 4, 32, 32).contiguous())
    assert torch.equal(y, y2) and torch.equal(last2, last.expand(1, 4, 32, 32))


@pytest.mark.parametrize("ragged, lengths", [(False, [1] * 9), (False, [40] * 3), (True, [500, 3, 0, 300]), (False, [900])])
def test_states_in_place(ragged, lengths):
    rows, n = sum(lengths), len(lengths)
    x, dy, d_last = inputs(rows, n, 4, 2, 64, 64, torch.bfloat16, seed=11)
    off = torch.tensor([0] + lengths, device="cuda").cumsum(0) if ragged else None
    att = gsr().LinearAttention(4, 64, 64, torch.bfloat16, kv_heads=2)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last, saved = att.forward(*args, state=x["state"], offsets=off, save=True)
    got = att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=off)
    state = x["state"].clone()
    y2, last2 = att.forward(*args, state=state, offsets=off, last=state)
    assert last2 is state and torch.equal(y, y2) and torch.equal(last, state)
    for target in (d_last, x["state"]):
        keep = {n_: torch.empty_like(got[n_]) for n_ in ("q", "k", "v", "gate")}
        want = target.clone()
        again = att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=off, grads={**keep, "state": target})
        for n_ in got:
            assert torch.equal(again[n_], got[n_]), n_
        target.copy_(want)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_tokens_one_by_one(dtype):
    """Single tokens on the carried state give what one pass over the sequences gives, each within its tolerance."""
    n, T, H, K, dk, dv = 30, 40, 4, 2, 64, 48
    x, _, _ = inputs(n * T, n, H, K, dk, dv, dtype, seed=12)
    att = gsr().LinearAttention(H, dk, dv, dtype, kv_heads=K)
    y, last = att.forward(x["q"], x["k"], x["v"], x["gate"], state=x["state"])
    state, out = x["state"].clone(), torch.empty_like(y)
    at = {m: x[m].view(n, T, *x[m].shape[1:]) for m in ("q", "k", "v", "gate")}
    for t in range(T):
        att.forward(*(at[m][:, t] for m in ("q", "k", "v", "gate")), state=state, last=state,
                    y=out.view(n, T, H, dv)[:, t])
    ref = ao.attention(x["q"], x["k"], x["v"], x["gate"], list(range(0, n * T + 1, T)), x["state"], dk ** -0.5)
    tol = tols(dtype, T)
    o.check(out, ref["y"], tol["y"], "tokens")
    o.check(state, ref["last"], tol["last"], "state")
    o.check(y, ref["y"], tol["y"], "pass")
    o.check(last, ref["last"], tol["last"], "last")


@pytest.mark.parametrize("width", [(1, 1), (64, 64), (33, 128), (128, 60), (128, 128)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_single_tokens(width, dtype):
    for gate in ("rows", "heads"):
        check_all(6, 2, *width, dtype, [1] * 11, False, gate=gate, seed=13)


def test_without_states():
    x, dy, _ = inputs(300, 1, 2, 2, 64, 64, torch.float32, seed=14)
    att = gsr().LinearAttention(2, 64, 64, torch.float32)
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last, saved = att.forward(*args, save=True)
    got = att.backward(*args, saved, dy)
    zero = torch.zeros(1, 2, 64, 64, device="cuda")
    ref = ao.attention(*args, [0, 300], zero, 0.125, dy, zero)
    tol = tols(torch.float32, 300)
    for n, t in {**got, "y": y, "last": last}.items():
        o.check(t, ref[n], tol[n], n)
    for n in ("q", "k", "v", "gate", "state"):  # each by itself
        only = att.backward(*args, saved, dy, grads={n: torch.empty_like(got[n])})
        assert set(only) == {n} and torch.equal(only[n], got[n]), n


def test_nothing_to_do():
    att = gsr().LinearAttention(2, 16, 16, torch.float32)
    x, _, _ = inputs(0, 3, 2, 2, 16, 16, torch.float32, gate="heads")
    args = (x["q"], x["k"], x["v"], x["gate"])
    y, last, saved = att.forward(*args, state=x["state"], save=True)
    assert y.shape == (0, 2, 16) and torch.equal(last, x["state"])
    d = torch.randn(3, 2, 16, 16, device="cuda")
    got = att.backward(*args, saved, y, d_last=d, state=x["state"])
    assert torch.equal(got["state"], d) and (got["gate"] == 0).all()
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    y, last = att.forward(*args, offsets=none)
    assert last.shape == (0, 2, 16, 16)


def test_offsets_out_of_range_are_not_followed():
    x, dy, d_last = inputs(300, 4, 2, 2, 32, 32, torch.bfloat16, seed=15)
    att = gsr().LinearAttention(2, 32, 32, torch.bfloat16)
    args = (x["q"], x["k"], x["v"], x["gate"])
    for bad in ([0, 400, 100, -5, 300], [7, 1 << 40, -(1 << 40), 250, 1 << 62], [300, 200, 100, 50, 0]):
        off = torch.tensor(bad, device="cuda")
        _, _, saved = att.forward(*args, state=x["state"], offsets=off, save=True)
        att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=off)
    torch.cuda.synchronize()
    good = torch.tensor([-3, 100, 150, 280, 900], device="cuda")  # clamped: 0 .. 300
    y, last = att.forward(*args, state=x["state"], offsets=good)
    y2, last2 = att.forward(*args, state=x["state"], offsets=torch.tensor([0, 100, 150, 280, 300], device="cuda"))
    assert torch.equal(y, y2) and torch.equal(last, last2)


def test_sequences_do_not_mix():
    """What is not a number in one sequence does not reach another."""
    x, dy, d_last = inputs(400, 4, 2, 2, 64, 64, torch.bfloat16, seed=16)
    off = torch.tensor([0, 90, 210, 211, 400], device="cuda")
    att = gsr().LinearAttention(2, 64, 64, torch.bfloat16)

    def run():
        args = (x["q"], x["k"], x["v"], x["gate"])
        y, last, saved = att.forward(*args, state=x["state"], offsets=off, save=True)
        return {**att.backward(*args, saved, dy, d_last=d_last, state=x["state"], offsets=off), "y": y, "last": last}

    want = run()
    for n, value in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("gate", float("nan"))):
        x[n][100:205] = value
    x["state"][1] = float("nan")
    got = run()
    for n in got:
        for a, b in ((0, 90), (210, 400)) if n in ("y", "q", "k", "v", "gate") else ((0, 1), (2, 4)):
            assert torch.equal(got[n][a:b], want[n][a:b]), n


def test_gradients_against_differences():
    """Central differences along random directions, in float32: the loss is a sum of about 1e4 terms of size 1, rounded
    to V each, over a step of 0.02: 1e-3 of the gradient's size covers that and the step's square."""
    x, dy, d_last = inputs(150, 2, 2, 1, 24, 24, torch.float32, seed=17, bias=1.0)
    off = torch.tensor([0, 20, 150], device="cuda")
    att = gsr().LinearAttention(2, 24, 24, torch.float32, kv_heads=1)
    order = ("q", "k", "v", "gate")
    _, _, saved = att.forward(*(x[n] for n in order), state=x["state"], offsets=off, save=True)
    got = att.backward(*(x[n] for n in order), saved, dy, d_last=d_last, state=x["state"], offsets=off)

    def loss(**new):
        t = {**x, **new}
        y, last = att.forward(*(t[n] for n in order), state=t["state"], offsets=off)
        return (y.double() * dy.double()).sum() + (last.double() * d_last.double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(18)
    for n, t in x.items():
        d = torch.randn(t.shape, generator=gen, device="cuda")
        slope = (loss(**{n: t + 0.01 * d}) - loss(**{n: t - 0.01 * d})) / 0.02
        assert abs(slope - (got[n].double() * d.double()).sum()) <= 1e-3 * got[n].double().norm() * d.double().norm(), n


@pytest.mark.parametrize("lengths", [[1] * 20, [700], [60] * 5])
def test_streams_and_graphs(lengths):
    rows, n = sum(lengths), len(lengths)
    x, dy, d_last = inputs(rows, n, 4, 2, 64, 64, torch.bfloat16, gate="heads", seed=19)
    att = gsr().LinearAttention(4, 64, 64, torch.bfloat16, kv_heads=2)
    args = (x["q"], x["k"], x["v"], x["gate"])

    def run(stream=None):
        y, last, saved = att.forward(*args, state=x["state"], save=True, stream=stream)
        return {**att.backward(*args, saved, dy, d_last=d_last, state=x["state"], stream=stream), "y": y, "last": last}

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (20, 21, 22):
        new, ndy, nd = inputs(rows, n, 4, 2, 64, 64, torch.bfloat16, gate="heads", seed=seed)
        for k in x:
            x[k].copy_(new[k])
        dy.copy_(ndy)
        d_last.copy_(nd)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(held[k], want[k]) for k in want)


def test_refusals():
    m = gsr()
    with pytest.raises(ValueError):
        m.LinearAttention(3, 16, 16, torch.float32, kv_heads=2)
    att = m.LinearAttention(2, 16, 16, torch.float32)
    x, _, _ = inputs(12, 3, 2, 2, 16, 16, torch.float32)
    args = [x["q"], x["k"], x["v"], x["gate"]]
    for i, bad in ((0, x["q"].half()), (0, x["q"][:, :1]), (1, x["k"][:11]), (2, x["v"].transpose(1, 2)),
                   (3, x["gate"].half()), (3, x["gate"][:, :1]), (3, x["gate"][0, :1]), (0, x["q"].cpu())):
        wrong = list(args)
        wrong[i] = bad
        with pytest.raises(ValueError):
            att.forward(*wrong)
    with pytest.raises(ValueError):
        att.forward(*args, state=x["state"].half())
    with pytest.raises(ValueError):
        att.forward(*args, offsets=torch.tensor([0, 12], dtype=torch.int32, device="cuda"))
    with pytest.raises(m.GsrError):
        att.forward(*args, state=x["state"][:1].expand(5, 2, 16, 16).contiguous())  # 12 rows are not 5 equal sequences
    with pytest.raises(m.GsrError):
        att.forward(*args, y=torch.empty(12, 1, 16, device="cuda").expand(12, 2, 16))
    with pytest.raises(m.GsrError):
        wide = m.LinearAttention(1, 129, 16, torch.float32)
        wide.forward(torch.zeros(4, 1, 129, device="cuda"), torch.zeros(4, 1, 129, device="cuda"),
                     torch.zeros(4, 1, 16, device="cuda"), torch.zeros(1, device="cuda"))
    y, last, saved = att.forward(*args, state=x["state"], save=True)
    states = torch.zeros(4, 2, 16, 16, device="cuda")
    with pytest.raises(m.GsrError):
        att.forward(*args, state=states[:3], last=states[1:])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("name", ["q", "k", "v", "gate"])
def test_earlier_rows_are_left_alone(name, dtype):
    """What is not a number reaches no row before its own, whatever tile they share."""
    x, _, _ = inputs(200, 1, 4, 2, 64, 72, dtype, seed=23)
    att = gsr().LinearAttention(4, 64, 72, dtype, kv_heads=2)
    run = lambda: att.forward(x["q"], x["k"], x["v"], x["gate"], state=x["state"])  # noqa: E731
    want, _ = run()
    at = 77
    if name == "gate":
        x[name][at, 1] = float("nan")
    else:
        x[name][at, -1, 5] = float("inf") if name == "v" else float("nan")
        if name == "v":
            x[name][at + 30, -1, 9] = float("nan")
    got, last = run()
    assert torch.equal(got[:at], want[:at])
    heads = slice(3, 4) if name == "q" else slice(2, 4)  # of the second key head, or the one query head
    other = slice(0, 3) if name == "q" else slice(0, 2)
    assert torch.equal(got[:, other], want[:, other])
    if name == "q":
        assert torch.isnan(got[at, heads]).all() and torch.equal(got[at + 1:], want[at + 1:])
    elif name == "v":
        assert not torch.isfinite(got[at:, heads, 5]).any() and torch.isnan(got[at + 30:, heads, 9]).all()
        rest = [c for c in range(72) if c not in (5, 9)]
        assert torch.equal(got[:, heads][..., rest], want[:, heads][..., rest])
        assert torch.equal(got[:at + 30, heads, 9], want[:at + 30, heads, 9])
        assert not torch.isfinite(last[0, 1, :, 5]).any() and torch.isfinite(last[0, 0]).all()
    else:
        assert torch.isnan(got[at:, heads]).all()
