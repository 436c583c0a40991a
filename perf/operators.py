"""The learned updater's operators, as they are measured: the gated feed-forward block,
the gated linear recurrence and the Newton-Schulz orthogonalisation, in plain torch
(`own = False`) and through the library (`own = True`)."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_NS = (3.4445, -4.7750, 2.0315)  # the quintic's coefficients


def _ffn(name, m, d_in, hidden, d_out, dtype, act, train):
    return {"name": name, "op": "ffn", "m": m, "d_in": d_in, "hidden": hidden, "d_out": d_out, "dtype": dtype,
            "act": act, "train": train}


def _scan(name, rows, channels, n_seq, ragged, dtype, train):
    return {"name": name, "op": "scan", "rows": rows, "channels": channels, "n_seq": n_seq, "ragged": ragged,
            "dtype": dtype, "train": train}


def _ortho(name, batch, rows, cols, dtype, out_dtype):
    return {"name": name, "op": "ortho", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype,
            "out_dtype": out_dtype, "steps": 5}


def listed():
    return [
        # one token through a wide block: the smallest call, bound by the weights' bytes
        _ffn("ffn_one_row", 1, 1024, 4096, 1024, "bf16", "silu", False),
        # a few dozen tokens of a small serving batch
        _ffn("ffn_small_batch", 48, 1024, 2816, 1024, "bf16", "silu", False),
        # degree-3 score tokens (57 wide) of a compact anchor scene (1,440 anchors x 16) in the tokens' own type
        _ffn("ffn_tokens_f32", 23040, 57, 256, 128, "f32", "gelu", True),
        # the updater's block on the same Gaussians, one training step
        _ffn("ffn_train", 23040, 512, 2048, 512, "bf16", "gelu", True),
        # odd sizes throughout, rows that are not 16-byte aligned
        _ffn("ffn_ragged_f16", 8191, 500, 1366, 500, "f16", "silu", True),
        # the updater's block over the pixel-aligned Gaussians of two 256 x 256 views: the largest
        _ffn("ffn_train_large", 131072, 512, 2048, 512, "bf16", "silu", True),
        # hidden state of every Gaussian of the 2,000-Gaussian scene advanced by one step
        _scan("scan_step", 2000, 256, 2000, False, "bf16", False),
        # all 311,296 Gaussians of the compact 512 x 960 scene as one depth-ordered sequence
        _scan("scan_long_train", 311296, 256, 1, False, "bf16", True),
        # scenes of different sizes packed one after another (some of them empty), in float32
        _scan("scan_ragged_f32", 50021, 192, 37, True, "f32", True),
        # the updater's small weight matrices, float32 momentum, one batch
        _ortho("ortho_small_batch", 12, 128, 512, "f32", "bf16"),
        # tall odd matrices, float32 throughout
        _ortho("ortho_odd_f32", 2, 1366, 500, "f32", "f32"),
        # one wide matrix, the largest
        _ortho("ortho_large", 1, 2048, 5632, "bf16", "bf16"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ffn", "scan", "ortho"))
    while True:
        if op == "ffn":
            dtype = rng.choice(("bf16", "f16", "f32"))
            train = rng.random() < 0.6
            c = _ffn("", _logint(rng, 1, 131072), _logint(rng, 32, 1024), _logint(rng, 32, 4096),
                     _logint(rng, 32, 1024), dtype, rng.choice(("silu", "gelu")), train)
            if rng.random() < 0.5:  # model widths are usually multiples of 64
                for k in ("d_in", "hidden", "d_out"):
                    c[k] = max(64, c[k] // 64 * 64)
            limit = 2.4e12 if dtype != "f32" else 2.4e11
        elif op == "scan":
            rows = _logint(rng, 64, 311296)
            ragged = rng.random() < 0.5
            n_seq = _logint(rng, 1, rows)
            if not ragged:
                rows = max(1, rows // n_seq) * n_seq
            c = _scan("", rows, _logint(rng, 32, 1024), n_seq, ragged, rng.choice(("bf16", "f16", "f32")),
                      rng.random() < 0.6)
            limit = 2.4e9 if c["train"] else 1.2e9
        else:
            dtype, out = rng.choice((("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")))
            c = _ortho("", rng.choice((1, 1, 2, 4, 12)), _logint(rng, 32, 5632), _logint(rng, 32, 5632), dtype, out)
            limit = 4.2e11 if out != "f32" else 1.5e11
            if min(c["rows"], c["cols"]) > 2048:
                continue
        if op == "scan":
            cost = c["rows"] * c["channels"] * (30 if c["train"] else 15)
        else:
            cost = work(c)["flops"]
        if cost <= limit and 48 * 64 not in c.values():
            return {k: v for k, v in c.items() if k != "name"}


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "ffn":
        m, d, f, o = case["m"], case["d_in"], case["hidden"], case["d_out"]
        weights = 2 * f * d + o * f
        nbytes = e * (m * d + weights + m * o)
        flops = 2 * m * f * (2 * d + o)
        if case["train"]:
            nbytes += e * (m * o + m * d + weights)
            flops *= 3
    elif case["op"] == "scan":
        n = case["rows"] * case["channels"]
        state = 4 * case["n_seq"] * case["channels"]
        nbytes = 3 * n * e + 2 * state
        flops = 9 * n
        if case["train"]:
            nbytes += 3 * n * e + 2 * state
            flops += 9 * n
        if case["ragged"]:
            nbytes += 8 * (case["n_seq"] + 1)
    else:
        lo, hi = sorted((case["rows"], case["cols"]))
        nbytes = case["batch"] * lo * hi * (e + _BYTES[case["out_dtype"]])
        # the two symmetric products need half of their entries
        flops = case["batch"] * case["steps"] * (3 * lo * lo * hi + lo ** 3)
    return {"bytes": nbytes, "flops": flops}


def _inputs(case, seed):
    """The tensors a caller holds, made on the GPU from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    if case["op"] == "ffn":
        m, d, f, o = case["m"], case["d_in"], case["hidden"], case["d_out"]
        t = {"x": normal(m, d), "w_gate": normal(f, d, scale=d ** -0.5), "w_up": normal(f, d, scale=d ** -0.5),
             "w_down": normal(o, f, scale=f ** -0.5)}
        if case["train"]:
            t["dy"] = normal(m, o)
    elif case["op"] == "scan":
        r, c, s = case["rows"], case["channels"], case["n_seq"]
        # forget gates biased towards keeping the state, as recurrent layers initialise them
        t = {"gate": (torch.randn(r, c, generator=gen, device="cuda") * 1.5 + 2.0).to(dt), "x": normal(r, c),
             "h0": normal(s, c, dtype=torch.float32)}
        if case["ragged"]:
            cuts = torch.randint(0, r + 1, (s - 1,), generator=gen, device="cuda").sort().values
            t["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), r)])
        else:
            t["offsets"] = None
        if case["train"]:
            t["dy"] = normal(r, c)
            t["dh_last"] = normal(s, c, dtype=torch.float32)
    else:
        t = {"g": normal(case["batch"], case["rows"], case["cols"], scale=0.02)}
    return t


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import gaussian_splatting_rasterizer_amd as gsr
        if case["op"] == "ffn":
            state["block"] = gsr.GatedFFN(state["w_gate"], state["w_up"], state["w_down"], activation=case["act"])
        elif case["op"] == "scan":
            state["scan"] = gsr.GatedScan(case["channels"], _DTYPES[case["dtype"]])
        else:
            state["ortho"] = gsr.Orthogonalizer(case["batch"], case["rows"], case["cols"], _DTYPES[case["dtype"]],
                                                _DTYPES[case["out_dtype"]], steps=case["steps"], coefficients=_NS)
    return state


def _run_own(s):
    case = s["case"]
    if case["op"] == "ffn":
        if not case["train"]:
            return s["block"].forward(s["x"])
        y, saved = s["block"].forward(s["x"], save=True)
        g = s["block"].backward(s["x"], saved, s["dy"])
        return y, g["x"], g["w_gate"], g["w_up"], g["w_down"]
    if case["op"] == "scan":
        if not case["train"]:
            return s["scan"].forward(s["gate"], s["x"], h0=s["h0"], offsets=s["offsets"])
        y, h_last, saved = s["scan"].forward(s["gate"], s["x"], h0=s["h0"], offsets=s["offsets"], save=True)
        g = s["scan"].backward(s["gate"], s["x"], saved, s["dy"], s["dh_last"], h0=s["h0"], offsets=s["offsets"])
        return y, h_last, g["gate"], g["x"], g["h0"]
    return s["ortho"].run(s["g"])


def _act(g, name):
    """Activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_ffn(s):
    case, dt = s["case"], s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, case["act"])
    h = a * u
    y = (h @ wd.t()).to(dt)
    if not case["train"]:
        return y
    dy = s["dy"].float()
    dh = dy @ wd
    du, dg = dh * a, dh * u * da
    dx = dg @ wg + du @ wu
    return y, dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ h).to(dt)


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0 from zero, by combining spans of doubling length."""
    n, k = a.shape[0], 1
    while k < n:
        b = torch.cat([b[:k], a[k:] * b[:-k] + b[k:]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _bounds(s, device):
    case = s["case"]
    if s["offsets"] is not None:
        return s["offsets"]
    return torch.arange(case["n_seq"] + 1, device=device) * (case["rows"] // case["n_seq"])


def _plain_scan(s):
    case, dt = s["case"], s["x"].dtype
    a, x, h0 = torch.sigmoid(s["gate"].float()), s["x"].float(), s["h0"]
    na = torch.sigmoid(-s["gate"].float())
    off = _bounds(s, x.device)
    idx = torch.searchsorted(off, torch.arange(x.shape[0], device=x.device), right=True) - 1  # each row's sequence
    first = (torch.arange(x.shape[0], device=x.device) == off[idx]).unsqueeze(1)
    b = na * x + torch.where(first, a * h0[idx], 0.0)
    keep = torch.where(first, 0.0, a)  # a sequence's first row forgets the row before it
    h = _doubling(keep, b)
    last = (off[1:] - 1).clamp(min=0)
    empty = (off[1:] == off[:-1]).unsqueeze(1)
    h_last = torch.where(empty, h0, h[last])
    if not case["train"]:
        return h.to(dt), h_last
    end = torch.arange(x.shape[0], device=x.device) == off[idx + 1] - 1
    up = s["dy"].float() + torch.where(end.unsqueeze(1), s["dh_last"][idx], 0.0)
    nxt = torch.cat([keep[1:], torch.zeros_like(keep[:1])])
    grad = _doubling(nxt.flip(0), up.flip(0)).flip(0)
    prev = torch.where(first, h0[idx], torch.cat([h[:1], h[:-1]]))
    start = off[:-1].clamp(max=x.shape[0] - 1)
    dh0 = torch.where(empty, s["dh_last"], a[start] * grad[start])
    return h.to(dt), h_last, (grad * (prev - x) * a * na).to(dt), (grad * na).to(dt), dh0


def _plain_ortho(s):
    case = s["case"]
    x = s["g"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / x.square().sum(dim=(1, 2), keepdim=True).sqrt().clamp(min=1e-7)
    a, b, c = _NS
    for _ in range(case["steps"]):
        p = torch.stack([m @ m.t() for m in x])
        q = torch.stack([b * m + c * (m @ m) for m in p])
        x = torch.stack([a * m + k @ m for m, k in zip(x, q)])
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.to(_DTYPES[case["out_dtype"]])


def run(state):
    if own:
        return _run_own(state)
    return {"ffn": _plain_ffn, "scan": _plain_scan, "ortho": _plain_ortho}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def _exact_ffn(case, t):
    m = case["m"]
    y, dx = [], []
    grads = {k: torch.zeros(t[k].shape, dtype=torch.float64, device="cuda") for k in ("w_gate", "w_up", "w_down")}
    w = {k: t[k].double() for k in grads}
    for r0 in range(0, m, 16384):  # blocks of rows
        x = t["x"][r0:r0 + 16384].double()
        gate = torch.mm(x, w["w_gate"].t())
        up = torch.mm(x, w["w_up"].t())
        if case["act"] == "silu":
            prob = 1.0 / (1.0 + torch.exp(-gate))
            slope = prob + gate * prob * (1.0 - prob)
        else:
            prob = torch.special.ndtr(gate)
            slope = prob + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
        hid = gate * prob * up
        y.append(torch.mm(hid, w["w_down"].t()))
        if case["train"]:
            dy = t["dy"][r0:r0 + 16384].double()
            dh = torch.mm(dy, w["w_down"])
            grads["w_down"] += torch.mm(dy.t(), hid)
            d_gate = dh * up * slope
            d_up = dh * gate * prob
            grads["w_gate"] += torch.mm(d_gate.t(), x)
            grads["w_up"] += torch.mm(d_up.t(), x)
            dx.append(torch.mm(d_gate, w["w_gate"]) + torch.mm(d_up, w["w_up"]))
    if not case["train"]:
        return torch.cat(y)
    return torch.cat(y), torch.cat(dx), grads["w_gate"], grads["w_up"], grads["w_down"]


def _blocked(a, b):
    """h_t = a_t h_{t-1} + b_t in sqrt(n) blocks: every block from zero, then the carries between them."""
    n, c = a.shape
    size = max(1, math.isqrt(n))
    blocks = -(-n // size)
    pad = blocks * size - n
    a = torch.cat([a, a.new_zeros(pad, c)]).view(blocks, size, c)
    b = torch.cat([b, b.new_zeros(pad, c)]).view(blocks, size, c)
    h, decay = torch.empty_like(b), torch.empty_like(a)
    h[:, 0], decay[:, 0] = b[:, 0], a[:, 0]
    for i in range(1, size):
        h[:, i] = a[:, i] * h[:, i - 1] + b[:, i]
        decay[:, i] = a[:, i] * decay[:, i - 1]
    carry = h.new_zeros(c)
    for k in range(blocks):
        h[k] += decay[k] * carry
        carry = h[k, -1]
    return h.view(-1, c)[:n]


def _exact_scan(case, t):
    n, s = case["rows"], case["n_seq"]
    if t["offsets"] is None:
        lengths = [n // s] * s
    else:
        lengths = (t["offsets"][1:] - t["offsets"][:-1]).tolist()
    starts, ends, rows = [], [], []
    at = 0
    for i, ln in enumerate(lengths):
        if ln:
            starts.append(at)
            ends.append(at + ln - 1)
            rows.append(i)
        at += ln
    starts, ends, rows = (torch.tensor(v, device="cuda") for v in (starts, ends, rows))
    z, x, h0 = t["gate"].double(), t["x"].double(), t["h0"].double()
    keep = 1 / (1 + torch.exp(-z))
    take = 1 / (1 + torch.exp(z))
    mul, add = keep.clone(), take * x
    mul[starts] = 0
    add[starts] += keep[starts] * h0[rows]
    h = _blocked(mul, add)
    h_last = h0.clone()
    h_last[rows] = h[ends]
    if not case["train"]:
        return h, h_last
    up = t["dy"].double()
    up[ends] += t["dh_last"].double()[rows]
    back = torch.zeros_like(mul)
    back[:-1] = mul[1:]
    g = _blocked(back.flip(0), up.flip(0)).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[starts] = h0[rows]
    dh0 = t["dh_last"].double()
    dh0[rows] = keep[starts] * g[starts]
    return h, h_last, g * keep * take * (before - x), g * take, dh0


def _exact_ortho(case, t):
    a, b, c = _NS
    out = []
    for m in t["g"].double():
        x = m / max(float(m.norm()), 1e-7)
        for _ in range(case["steps"]):  # the quintic applied on the smaller side
            if case["rows"] > case["cols"]:
                p = x.t() @ x
                x = a * x + x @ (b * p + c * (p @ p))
            else:
                p = x @ x.t()
                x = a * x + (b * p + c * (p @ p)) @ x
        out.append(x)
    return torch.stack(out)


def exact(case, seed):
    return {"ffn": _exact_ffn, "scan": _exact_scan, "ortho": _exact_ortho}[case["op"]](case, _inputs(case, seed))
