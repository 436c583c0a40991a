"""More of the learned updater's operators, as they are measured: linear attention with a decay for each head, the
root-mean-square norm with the residual's addition and the AdamW step over many tensors, in plain torch (`own = False`)
and through the library (`own = True`)."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_F8 = torch.float8_e4m3fn
_F8_MAX, _F8_MIN = 448.0, 2.0 ** -9
_BLOCK = 256  # values that share a scale of the optimizer's 8-bit states
_EPS = 1e-6
_BETAS, _ADAM_EPS, _STEPS_DONE = (0.9, 0.999), 1e-8, 99


def _attn(name, rows, n_seq, ragged, heads, kv_heads, d_key, d_value, dtype, train, gate):
    """gate: "rows" (one value for each row and head, float32) or "heads" (one for each head)."""
    return {"name": name, "op": "attn", "rows": rows, "n_seq": n_seq, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "d_key": d_key, "d_value": d_value, "dtype": dtype, "train": train, "gate": gate}


def _norm(name, rows, width, dtype, stream, train, group):
    """stream: the type of the residual; group: columns that share a scale of the 8-bit output (0: the row), -1 where
    the output is of the input's type."""
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "stream": stream, "train": train,
            "group": group}


def _adam(name, kind, count, dtype, grad, copy, bits):
    """kind "scene": the five parameter tensors of `count` Gaussians; "weights": the six matrices of an updater `count`
    channels wide.  copy: the type of the copies that the step writes beside the parameters ("" for none)."""
    return {"name": name, "op": "adam", "kind": kind, "count": count, "dtype": dtype, "grad": grad, "copy": copy,
            "bits": bits}


def listed():
    return [
        # one token for each of a few sequences with a wide state: the smallest call of the attention
        _attn("attn_step_few", 48, 48, False, 8, 2, 128, 128, "bf16", False, "rows"),
        # the memory of every Gaussian of the 2,000-Gaussian scene advanced by one token
        _attn("attn_step", 2000, 2000, False, 4, 4, 64, 64, "bf16", False, "rows"),
        # all 311,296 Gaussians of the compact 512 x 960 scene as one depth-ordered sequence
        _attn("attn_long", 311296, 1, False, 4, 4, 64, 64, "bf16", False, "heads"),
        # training on the Gaussians of two 256 x 256 views, the block's 512 channels: the attention's largest
        _attn("attn_train_large", 131072, 1, False, 4, 4, 128, 128, "bf16", True, "rows"),
        # the 1,440 anchors of a compact scene, the 16 Gaussians of each a short sequence with a first state
        _attn("attn_anchors_f16", 23040, 1440, False, 4, 2, 64, 64, "f16", True, "rows"),
        # scenes of different sizes packed one after another (some of them empty), odd widths, float32
        _attn("attn_ragged_f32", 50021, 37, True, 6, 2, 57, 72, "f32", True, "heads"),
        # a few dozen tokens of a small serving batch: the smallest call of the norm
        _norm("norm_small_batch", 48, 1024, "bf16", "bf16", False, -1),
        # in front of the updater's block over the Gaussians of two 256 x 256 views, float32 residual, one training step
        _norm("norm_train", 131072, 512, "bf16", "f32", True, -1),
        # the same rows kept in 8 bits
        _norm("norm_8bit", 131072, 512, "bf16", "bf16", False, 128),
        # the weights of the example's updater and the copies its products read: the smallest call of the step
        _adam("adam_weights", "weights", 64, "f32", "bf16", "bf16", 32),
        # the parameters of the compact 512 x 960 scene
        _adam("adam_scene", "scene", 311296, "f32", "f32", "", 32),
        # the parameters of the dense 512 x 960 scene, states in 8 bits: the largest
        _adam("adam_scene_8bit", "scene", 5898240, "f32", "f32", "", 8),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "norm", "adam"))
    while True:
        if op == "attn":
            shape = rng.choice(("step", "one", "equal", "ragged"))
            train = shape != "step" and rng.random() < 0.6
            kv = rng.choice((1, 2, 3, 4, 8))
            heads = kv * rng.choice((1, 1, 2, 3, 4))
            if rng.random() < 0.5:
                dk, dv = rng.choice(((64, 64), (128, 128), (64, 128), (128, 64), (32, 32)))
            else:
                dk, dv = rng.randint(16, 128), rng.randint(16, 128)
            rows = _logint(rng, 1, 2000) if shape == "step" else _logint(rng, 64, 311296)
            n_seq = {"step": rows, "one": 1}.get(shape) or _logint(rng, 2, min(rows, 4000))
            if shape == "equal":
                rows = rows // n_seq * n_seq
            c = _attn("", rows, n_seq, shape == "ragged", heads, kv, dk, dv, rng.choice(("bf16", "f16", "f32")), train,
                      rng.choice(("rows", "rows", "heads")))
            w = work(c)
            fits = w["bytes"] <= 1.0e9 and w["flops"] <= 1.6e11
        elif op == "norm":
            dtype = rng.choice(("bf16", "f16", "f32"))
            train = rng.random() < 0.5
            width = _logint(rng, 33, 8192)
            if rng.random() < 0.5:  # model widths are usually multiples of 64
                width = max(64, width // 64 * 64)
            c = _norm("", _logint(rng, 1, 131072), width, dtype, rng.choice((dtype, "f32")), train,
                      -1 if train else rng.choice((-1, -1, 0, 32, 64, 128)))
            fits = work(c)["bytes"] <= 1.0e9
        else:
            kind = rng.choice(("scene", "weights"))
            dtype = rng.choice(("f32", "f32", "bf16", "f16"))
            c = _adam("", kind, _logint(rng, 1, 5898240) if kind == "scene" else _logint(rng, 8, 4096), dtype,
                      rng.choice((dtype, "f32", "bf16")), rng.choice(("", "", "bf16", "f16")), rng.choice((32, 8)))
            fits = work(c)["bytes"] <= 6.4e9
        if fits:
            return {k: v for k, v in c.items() if k != "name"}


def _shapes(case):
    n = case["count"]
    if case["kind"] == "scene":  # means, quaternions, scales, opacities, colours of degree 3
        return [(n, 3), (n, 4), (n, 3), (n,), (n, 16, 3)]
    hidden, token, params = 4 * n, 57, 59
    return [(hidden, token), (hidden, token), (2 * n, hidden), (hidden, n), (hidden, n), (params, hidden)]


def work(case):
    if case["op"] == "attn":
        e, r, kv, h = _BYTES[case["dtype"]], case["rows"], case["kv_heads"], case["heads"]
        dk, dv, train = case["d_key"], case["d_value"], case["train"]
        tokens = e * r * (h + kv) * (dk + dv)
        gate = 4 * kv * (r if case["gate"] == "rows" else 1)
        states = 2 * 4 * case["n_seq"] * kv * dk * dv
        # a token reads the state and is added to it; backward: three products with the states, and both of them built
        flops = 2 * r * dk * dv * ((kv + h) if not train else (kv + h) + (2 * h + 3 * kv))
        # backward: the gradient of the outputs and of every input
        nbytes = tokens + gate + states
        if train:
            nbytes += e * r * (h * dv + h * dk + kv * (dk + dv)) + gate + states
        if case["ragged"]:
            nbytes += 8 * (case["n_seq"] + 1)
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "norm":
        e, s, n = _BYTES[case["dtype"]], _BYTES[case["stream"]], case["rows"] * case["width"]
        out = e * n
        if case["group"] >= 0:
            out = n + 4 * case["rows"] * (-(-case["width"] // case["group"]) if case["group"] else 1)
        nbytes = n * (e + 2 * s) + out + 4 * case["width"]
        if case["train"]:  # gradients of the output and of the new residual; of the input, the residual and the weight
            nbytes += n * (e + s + s + (e if e != s else 0)) + 4 * case["width"]
        return {"bytes": nbytes, "flops": (18 if case["train"] else 7) * n}
    n = sum(math.prod(s) for s in _shapes(case))
    states = 16 * n if case["bits"] == 32 else 4 * n + 16 * (n // _BLOCK)
    copy = _BYTES[case["copy"]] if case["copy"] else 0
    return {"bytes": n * (2 * _BYTES[case["dtype"]] + _BYTES[case["grad"]] + copy) + states, "flops": 15 * n}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _attn_inputs(case, seed):
    gen, dt = _gen(seed), _DTYPES[case["dtype"]]
    r, h, kv, dk, dv, n = (case[k] for k in ("rows", "heads", "kv_heads", "d_key", "d_value", "n_seq"))

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    t = {"q": normal(r, h, dk), "k": normal(r, kv, dk, scale=dk ** -0.5), "v": normal(r, kv, dv)}
    if case["gate"] == "rows":  # biased towards keeping the state, as recurrent layers initialise them
        t["gate"] = torch.randn(r, kv, generator=gen, device="cuda") * 1.5 + 3.0
    else:  # memories of 16 rows and longer, a factor of two from head to head
        t["gate"] = 2.7 + 0.7 * torch.arange(kv, device="cuda") + torch.rand(kv, generator=gen, device="cuda") * 0.1
    t["state"] = normal(n, kv, dk, dv, dtype=torch.float32)
    t["offsets"] = None
    if case["ragged"]:
        cuts = torch.randint(0, r + 1, (n - 1,), generator=gen, device="cuda").sort().values
        t["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), r)])
    if case["train"]:
        t["dy"] = normal(r, h, dv)
        t["d_last"] = normal(n, kv, dk, dv, scale=0.1, dtype=torch.float32)
    return t


def _norm_inputs(case, seed):
    gen, dt, st = _gen(seed), _DTYPES[case["dtype"]], _DTYPES[case["stream"]]
    r, w = case["rows"], case["width"]
    t = {"x": torch.randn(r, w, generator=gen, device="cuda").to(dt),
         "residual": (torch.randn(r, w, generator=gen, device="cuda") * 3).to(st),
         "weight": 1 + 0.1 * torch.randn(w, generator=gen, device="cuda")}
    if case["train"]:
        t["dy"] = torch.randn(r, w, generator=gen, device="cuda").to(dt)
        t["dh"] = torch.randn(r, w, generator=gen, device="cuda").to(st)
    return t


def _codes(x, nonzero=False):
    """8-bit values and scales of blocks of 256, in the type of x."""
    blocks = torch.nn.functional.pad(x, (0, -x.numel() % _BLOCK)).view(-1, _BLOCK)
    top = blocks.abs().amax(dim=1, keepdim=True)
    scale = torch.where(top > 0, top / _F8_MAX, torch.ones_like(top))
    c = blocks / scale
    if nonzero:  # what is not zero does not become zero
        c = torch.where(c > 0, c.clamp(min=_F8_MIN), c)
    return c.to(_F8).view(-1)[:x.numel()], scale.view(-1).float()


def _values(code, scale, dtype):
    return code.to(dtype) * scale.to(dtype).repeat_interleave(_BLOCK)[:code.numel()]


def _adam_inputs(case, seed):
    gen, dt, gt = _gen(seed), _DTYPES[case["dtype"]], _DTYPES[case["grad"]]
    t = {"p": [], "g": [], "m": [], "v": [], "m_scale": [], "v_scale": []}
    for shape in _shapes(case):
        n = math.prod(shape)
        t["p"].append(torch.randn(shape, generator=gen, device="cuda").to(dt))
        # gradients of very different sizes, and some that are zero: a Gaussian that no view sees
        size = torch.exp(2 * torch.randn(n, generator=gen, device="cuda")) * 1e-3
        g = torch.randn(n, generator=gen, device="cuda") * size
        g = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.2, torch.zeros_like(g), g)
        t["g"].append(g.to(gt).view(shape))
        m = torch.randn(n, generator=gen, device="cuda") * size * 0.3
        v = size.square() * (0.5 + torch.rand(n, generator=gen, device="cuda")) * (1 - _BETAS[1] ** _STEPS_DONE)
        if case["bits"] == 32:
            t["m"].append(m)
            t["v"].append(v)
            continue
        for key, x in (("m", m), ("v", v.sqrt())):  # v is held as its root
            code, scale = _codes(x, key == "v")
            t[key].append(code)
            t[key + "_scale"].append(scale)
    t["rates"] = [1.6e-4, 1e-3, 5e-3, 5e-2, 2.5e-3] if case["kind"] == "scene" else [1e-3] * 6
    return t


def prepare(case, seed):
    s = {"attn": _attn_inputs, "norm": _norm_inputs, "adam": _adam_inputs}[case["op"]](case, seed)
    s["case"] = case
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "adam":
        s["steps"] = torch.full((), _STEPS_DONE, dtype=torch.int64, device="cuda")
        s["copies"] = [p.to(_DTYPES[case["copy"]], copy=True) for p in s["p"]] if case["copy"] else None
    if own:
        import gaussian_splatting_rasterizer_amd as gsr
        if case["op"] == "attn":
            s["attn"] = gsr.LinearAttention(case["heads"], case["d_key"], case["d_value"], dt,
                                            kv_heads=case["kv_heads"])
        elif case["op"] == "norm":
            s["norm"] = gsr.ResidualNorm(s["weight"], dt, eps=_EPS)
        else:
            opt = gsr.AdamW(s["p"], lr=s["rates"], betas=_BETAS, eps=_ADAM_EPS, weight_decay=0.01,
                            state_bits=case["bits"], copies=s["copies"])
            opt.steps.fill_(_STEPS_DONE)
            for key, mine in (("m", opt.m), ("v", opt.v), ("m_scale", opt.m_scale), ("v_scale", opt.v_scale)):
                for given, t in zip(s.pop(key), mine):
                    t.copy_(given)
            s["opt"] = opt
    return s


def _run_own(s):
    case = s["case"]
    if case["op"] == "attn":
        a = (s["q"], s["k"], s["v"], s["gate"])
        if not case["train"]:
            return s["attn"].forward(*a, state=s["state"], offsets=s["offsets"])
        y, last, saved = s["attn"].forward(*a, state=s["state"], offsets=s["offsets"], save=True)
        g = s["attn"].backward(*a, saved, s["dy"], d_last=s["d_last"], state=s["state"], offsets=s["offsets"])
        return y, last, g["q"], g["k"], g["v"], g["gate"], g["state"]
    if case["op"] == "norm":
        if case["group"] >= 0:
            return s["norm"].forward8(s["x"], s["residual"], group=case["group"])
        y, h = s["norm"].forward(s["x"], s["residual"])
        if not case["train"]:
            return y, h
        g = s["norm"].backward(h, s["dy"], s["dh"])
        return y, h, g["x"], g["residual"], g["weight"]
    opt = s["opt"]
    opt.step(s["g"])
    return s["p"], s["copies"], opt.m, opt.v, opt.m_scale, opt.v_scale


# ---- plain forms -------------------------------------------------------------------------------------------

def _doubling(a, b):
    """x_n = a_n x_{n-1} + b_n along dim 0 from zero, by combining spans of doubling length."""
    n, k = a.shape[0], 1
    while k < n:
        b = torch.cat([b[:k], a[k:] * b[:-k] + b[k:]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _chunks(s, size):
    """Rows of every chunk [n, size], which of them are rows, each chunk's sequence, and whether it is the first and
    the last of its sequence.  Chunks that the sequences do not need come last, with no rows."""
    case, dev = s["case"], s["q"].device
    off = s["offsets"]
    if off is None:
        off = torch.arange(case["n_seq"] + 1, device=dev) * (case["rows"] // case["n_seq"])
        n = case["n_seq"] * -(-(case["rows"] // case["n_seq"]) // size)
    else:
        n = case["rows"] // size + case["n_seq"]
    count = (off[1:] - off[:-1] + size - 1) // size
    end = count.cumsum(0)
    c = torch.arange(n, device=dev)
    seq = torch.searchsorted(end, c, right=True).clamp(max=case["n_seq"] - 1)
    nth = c - (end - count)[seq]
    row = (off[seq] + nth * size).unsqueeze(1) + torch.arange(size, device=dev)
    real = row < off[seq + 1].unsqueeze(1)
    used = c < end[-1]
    return row.clamp(max=case["rows"] - 1), real, seq, (nth == 0) & used, (nth == count[seq] - 1) & used, used


def _spread(t, row, real):
    """[rows, heads, d] -> [chunks, heads, size, d], zero where there is no row."""
    return (t.float()[row] * real[..., None, None]).permute(0, 2, 1, 3).contiguous()


def _plain_attn(s):
    case, dt = s["case"], s["q"].dtype
    r, hq, kv, dk, dv, n_seq = (case[k] for k in ("rows", "heads", "kv_heads", "d_key", "d_value", "n_seq"))
    G, scale = hq // kv, dk ** -0.5
    C = min(64, r // n_seq) if s["offsets"] is None else 64
    row, real, seq, first, last, used = _chunks(s, C)
    n = row.shape[0]
    q = _spread(s["q"], row, real).view(n, kv, G * C, dk)
    k, v = _spread(s["k"], row, real), _spread(s["v"], row, real)
    z = s["gate"].double()
    z = z[row] if z.dim() == 2 else z.expand(n, C, kv)
    p = (torch.nn.functional.logsigmoid(z) * real[..., None]).permute(0, 2, 1).cumsum(2)  # [n, kv, C], 64 bits
    low = torch.ones(C, C, dtype=torch.bool, device=p.device).tril()
    pair = torch.where(low, torch.exp(torch.where(low, p[..., :, None] - p[..., None, :], 0.0)), 0.0).float()
    into, out, through = (torch.exp(x).float() for x in (p, p[..., -1:] - p, p[..., -1]))
    through = through[..., None, None]
    fresh = first[:, None, None, None]
    first_of = torch.where(first, seq, n_seq)  # the chunk's sequence where it starts one
    prev = torch.arange(n, device=p.device).sub(1).clamp(min=0)
    grow = k.transpose(2, 3).contiguous() @ (v * out[..., None])
    before = _doubling(torch.where(fresh, 0.0, through[prev]),
                       torch.where(fresh, s["state"][seq], grow[prev] * used[:, None, None, None]))
    after = through * before + grow
    ends = torch.where(last, seq, n_seq)
    y_last = torch.cat([s["state"], s["state"][:1]])
    y_last = y_last.index_put((ends,), torch.where(last[:, None, None, None], after, 0.0))[:n_seq]

    def wide(x):  # the same for each query head of a group
        return x[:, :, None].expand(n, kv, G, *x.shape[2:]).reshape(n, kv, G * x.shape[2], *x.shape[3:])

    def gather(x, heads, d):  # [n, heads, C, d] -> [rows, heads, d]
        flat = x.view(n, heads, C, d).permute(0, 2, 1, 3).reshape(n * C, heads, d)
        at = torch.where(real, row, r).view(-1)
        return torch.zeros(r + 1, heads, d, device=x.device).index_copy_(0, at, flat)[:r]

    kt = k.transpose(2, 3).contiguous()
    scores = (q @ kt) * scale
    wpair, winto = wide(pair), wide(into)[..., None]
    y = (scores * wpair) @ v + winto * (q @ before) * scale
    y = gather(y, hq, dv).to(dt)
    if not case["train"]:
        return y, y_last
    do = _spread(s["dy"], row, real).view(n, kv, G * C, dv)
    qt = (q * winto * scale).transpose(2, 3).contiguous()
    shrink = qt @ do
    nxt = torch.arange(n, device=p.device).add(1).clamp(max=n - 1)
    lastd = last[:, None, None, None]
    at_end = _doubling(torch.where(lastd, 0.0, through[nxt]).flip(0),
                       torch.where(lastd, s["d_last"][seq], shrink[nxt] * used[nxt, None, None, None]).flip(0)).flip(0)
    at_start = through * at_end + shrink
    d_state = torch.cat([s["d_last"], s["d_last"][:1]])
    d_state = d_state.index_put((first_of,), torch.where(fresh, at_start, 0.0))[:n_seq]
    vt = v.transpose(2, 3).contiguous()
    dscores = (do @ vt) * wpair * scale
    rinter = winto * scale * (do @ before.transpose(2, 3).contiguous())
    dq = dscores @ k + rinter
    cinter = out[..., None] * (v @ at_end.transpose(2, 3).contiguous())
    dk_ = dscores.transpose(2, 3).contiguous() @ q + cinter
    dv_ = (scores * wpair).transpose(2, 3).contiguous() @ do + out[..., None] * (k @ at_end)
    # the pairs of a row at or behind t and a row before t: within the chunk, into it, out of it and across it
    W = (dscores * scores / scale).view(n, kv, G, C, C).sum(2) * ~torch.eye(C, dtype=torch.bool, device=p.device)
    W = W.flip(2).cumsum(2).flip(2).cumsum(3)  # [i >= t, j <= t']
    inside = torch.nn.functional.pad(W, (1, 0))[..., :C].diagonal(dim1=2, dim2=3)
    come = (rinter * q).sum(-1).view(n, kv, G, C).sum(2).flip(2).cumsum(2).flip(2)
    leave = (cinter * k).sum(-1)
    leave = leave.cumsum(2) - leave
    dg = inside + come + leave + (through * at_end * before).sum((2, 3))[..., None]
    dz = gather(dg[..., None], kv, 1)[..., 0] * torch.sigmoid(-s["gate"])
    if case["gate"] == "heads":
        dz = dz.double().sum(0).float()
    return (y, y_last, gather(dq, hq, dk).to(dt), gather(dk_, kv, dk).to(dt), gather(dv_, kv, dv).to(dt), dz, d_state)


def _plain_norm(s):
    case, dt, st = s["case"], s["x"].dtype, s["residual"].dtype
    h = s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS)
    y = h * rstd * s["weight"]
    kept = h.to(st)
    if case["group"] >= 0:
        rows, width = y.shape
        group = case["group"] or width
        parts = torch.nn.functional.pad(y, (0, -width % group)).view(rows, -1, group)
        top = parts.abs().amax(2, keepdim=True)
        scale = torch.where(top > 0, top / _F8_MAX, 1.0)
        return (parts / scale).to(_F8).view(rows, -1)[:, :width], scale[..., 0], kept
    if not case["train"]:
        return y.to(dt), kept
    # the gradients are those at the residual that was kept
    hk = kept.float()
    rstd = torch.rsqrt(hk.square().mean(1, keepdim=True) + _EPS)
    n, dy = hk * rstd, s["dy"].float()
    wdy = dy * s["weight"]
    dh = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True)) + s["dh"].float()
    return y.to(dt), kept, dh.to(dt), dh.to(st), (dy * n).double().sum(0).float()


def _plain_adam(s):
    case = s["case"]
    s["steps"] += 1
    t = s["steps"].double()
    b1, b2 = _BETAS
    c1, c2 = ((1 - b ** t).float() for b in _BETAS)
    for i, rate in enumerate(s["rates"]):
        p, g = s["p"][i].float().view(-1), s["g"][i].float().view(-1)
        if case["bits"] == 32:
            m, v = s["m"][i], s["v"][i]
        else:
            m = _values(s["m"][i], s["m_scale"][i], torch.float32)
            v = _values(s["v"][i], s["v_scale"][i], torch.float32).square()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        p = p - rate * 0.01 * p - rate * (m / c1) / (torch.sqrt(v / c2) + _ADAM_EPS)
        s["p"][i].copy_(p.view(s["p"][i].shape))
        if s["copies"]:
            s["copies"][i].copy_(p.view(s["p"][i].shape))
        if case["bits"] == 32:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
        else:
            for key, x in (("m", m), ("v", torch.sqrt(v))):
                code, scale = _codes(x, key == "v")
                s[key][i].copy_(code)
                s[key + "_scale"][i].copy_(scale)
    return s["p"], s["copies"], s["m"], s["v"], s["m_scale"], s["v_scale"]


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "norm": _plain_norm, "adam": _plain_adam}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def _exact_attn(case, seed):
    """Blocks of rows one after another, every sequence by itself (short ones of equal length at once), gradients by
    differentiation."""
    t = _attn_inputs(case, seed)
    n, G = case["n_seq"], case["heads"] // case["kv_heads"]
    off = t["offsets"]
    if off is None:
        parts = [(0, case["rows"], n)]
        length = case["rows"] // n
    else:
        off = off.tolist()
        if n > 400:
            return None
        parts = [(off[i], off[i + 1], 1) for i in range(n)]
    names = ("q", "k", "v", "gate", "state")
    leaf = {k: t[k].double().requires_grad_(case["train"]) for k in names}
    grads = {k: torch.zeros_like(leaf[k]) for k in names}
    ys, lasts = [], []
    for s, (lo, hi, batch) in enumerate(parts):
        length = (hi - lo) // batch
        state0 = leaf["state"] if batch == n else leaf["state"][s:s + 1]
        S = state0
        outs = []

        def rows(x):  # blocks of [batch, heads, rows, d]
            x = x[lo:hi].view(batch, length, *x.shape[1:]).transpose(1, 2)
            return x.split(128, 2) if length else ()

        if case["gate"] == "rows":
            gates = [g[..., 0] for g in rows(leaf["gate"].unsqueeze(2))]
        else:
            gates = [leaf["gate"][None, :, None].expand(batch, case["kv_heads"], min(128, length - a))
                     for a in range(0, length, 128)]
        for q, k, v, g in zip(rows(leaf["q"]), rows(leaf["k"]), rows(leaf["v"]), gates):
            size = q.shape[2]
            c = torch.cumsum(-torch.log1p(torch.exp(-g)), 2)
            future = torch.ones(size, size, dtype=torch.bool, device="cuda").triu(1)
            decay = torch.exp((c.unsqueeze(3) - c.unsqueeze(2)).masked_fill(future, -math.inf))
            q = q.reshape(batch, case["kv_heads"], G, size, -1)
            att = torch.matmul(q, k.unsqueeze(2).transpose(3, 4)) * decay.unsqueeze(2)
            o = torch.matmul(att, v.unsqueeze(2)) + torch.matmul(q * torch.exp(c)[:, :, None, :, None], S.unsqueeze(2))
            outs.append(o.reshape(batch, case["heads"], size, -1).transpose(1, 2) * case["d_key"] ** -0.5)
            tail = torch.exp(c[..., -1:] - c).unsqueeze(3)
            S = S * torch.exp(c[..., -1])[..., None, None] + torch.matmul((k * tail).transpose(2, 3), v)
        y = torch.cat(outs, 1).reshape(hi - lo, case["heads"], -1) if outs else leaf["q"].new_zeros(0, case["heads"],
                                                                                                    case["d_value"])
        if case["train"]:
            d_last = t["d_last"].double()
            d_last = d_last if batch == n else d_last[s:s + 1]
            loss = (S * d_last).sum()
            if outs:
                loss = loss + (y * t["dy"][lo:hi].double()).sum()
            for key, g in zip(names, torch.autograd.grad(loss, [leaf[x] for x in names], allow_unused=True)):
                if g is not None:
                    grads[key] += g
        ys.append(y.detach())
        lasts.append(S.detach())
    y, last = torch.cat(ys), torch.cat(lasts)
    if not case["train"]:
        return y, last
    return y, last, grads["q"], grads["k"], grads["v"], grads["gate"], grads["state"]


def _round8(x):
    """The nearest 8-bit value (4 significant bits, at least 2^-9, at most 448), the even one of two, in 64 bits."""
    step = torch.exp2((torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4).double())
    return (x / step).round() * step


def _exact_norm(case, seed):
    t = _norm_inputs(case, seed)
    h = t["x"].double() + t["residual"].double()
    w = t["weight"].double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS) * w
    if case["group"] >= 0:
        codes, scales = [], []
        step = case["group"] or case["width"]
        for lo in range(0, case["width"], step):
            part = y[:, lo:lo + step]
            top = part.abs().max(1, keepdim=True).values / _F8_MAX
            top = torch.where(top > 0, top, 1.0)
            codes.append(_round8(part / top))
            scales.append(top)
        return torch.cat(codes, 1), torch.cat(scales, 1), h
    if not case["train"]:
        return y, h
    kept = h.to(_DTYPES[case["stream"]]).double()  # what the backward pass is given
    dy, width = t["dy"].double(), case["width"]
    inv = ((kept * kept).sum(1, keepdim=True) / width + _EPS) ** -0.5
    unit = kept * inv
    dunit = dy * w
    dh = t["dh"].double() + inv * (dunit - unit * ((dunit * unit).sum(1, keepdim=True) / width))
    return y, h, dh, dh, (dy * unit).sum(0)


def _exact_adam(case, seed):
    t = _adam_inputs(case, seed)
    out = {k: [] for k in ("p", "copies", "m", "v", "m_scale", "v_scale")}
    k = _STEPS_DONE + 1
    for i, rate in enumerate(t["rates"]):
        p, g = t["p"][i].double().flatten(), t["g"][i].double().flatten()
        if case["bits"] == 8:
            m, root = (_values(t[x][i], t[x + "_scale"][i], torch.float64) for x in ("m", "v"))
            v = root ** 2
        else:
            m, v = t["m"][i].double(), t["v"][i].double()
        m = m + (1 - _BETAS[0]) * (g - m)
        v = v + (1 - _BETAS[1]) * (g ** 2 - v)
        step = m / (1 - _BETAS[0] ** k) / ((v / (1 - _BETAS[1] ** k)) ** 0.5 + _ADAM_EPS)
        p = (p * (1 - 0.01 * rate) - rate * step).view(t["p"][i].shape)
        out["p"].append(p)
        if case["copy"]:
            out["copies"].append(p)
        if case["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
            continue
        for key, x in (("m", m), ("v", v ** 0.5)):
            code, scale = [], []
            for part in x.split(_BLOCK * 65536):
                whole = torch.zeros(-(-part.numel() // _BLOCK) * _BLOCK, dtype=torch.float64, device="cuda")
                whole[:part.numel()] = part
                whole = whole.view(-1, _BLOCK)
                top = whole.abs().max(1, keepdim=True).values / _F8_MAX
                top = torch.where(top > 0, top, 1.0)
                u = whole / top
                if key == "v":
                    u = torch.where((u > 0) & (u < _F8_MIN), _F8_MIN, u)
                code.append(_round8(u).flatten()[:part.numel()])
                scale.append(top.flatten())
            out[key].append(torch.cat(code))
            out[key + "_scale"].append(torch.cat(scale))
    return tuple(out[x] if out[x] or x != "copies" else None for x in out)


def exact(case, seed):
    return {"attn": _exact_attn, "norm": _exact_norm, "adam": _exact_adam}[case["op"]](case, seed)
