"""The updater's operators from their definitions, in float64 (numpy where small, torch float64 on the GPU for the
larger products).  Shared by the tests; it uses nothing of the package."""
import math

import numpy as np
import torch

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # 2^-(significant bits)


def act(g, name):
    """(act(g), act'(g)) in float64."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    cdf = torch.special.ndtr(g)
    return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def ffn(x, wg, wu, wd, name, dy=None):
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    a, da = act(g, name)
    h = a * u
    y = h @ wd.T
    if dy is None:
        return y
    dy = dy.double()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"y": y, "x": dg @ wg + du @ wu, "w_gate": dg.T @ x, "w_up": du.T @ x, "w_down": dy.T @ h}


def scan(gate, x, offsets, h0, dy=None, dh_last=None):
    """Row by row in numpy float64; offsets: list of n_seq + 1 row numbers."""
    gate, x, h0 = (np.asarray(t, np.float64) for t in (gate, x, h0))
    with np.errstate(over="ignore"):
        a, na = 1 / (1 + np.exp(-gate)), 1 / (1 + np.exp(gate))
    y, h_last, prev = np.zeros_like(x), h0.copy(), np.zeros_like(x)
    for s in range(len(offsets) - 1):
        h = h0[s].copy()
        for t in range(offsets[s], offsets[s + 1]):
            prev[t] = h
            h = a[t] * h + na[t] * x[t]
            y[t] = h
        h_last[s] = h
    if dy is None:
        return {"y": y, "h_last": h_last}
    dy, dh_last = np.asarray(dy, np.float64), np.asarray(dh_last, np.float64)
    dz, dx, dh0 = np.zeros_like(x), np.zeros_like(x), dh_last.copy()
    for s in range(len(offsets) - 1):
        e = dh_last[s].copy()
        for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
            G = dy[t] + e
            dx[t] = na[t] * G
            dz[t] = a[t] * na[t] * (prev[t] - x[t]) * G
            e = a[t] * G
        dh0[s] = e
    return {"y": y, "h_last": h_last, "gate": dz, "x": dx, "h0": dh0}


def newton_schulz(g, steps, coef, eps=1e-7):
    """One matrix, float64."""
    a, b, c = coef
    x = g.double()
    x = x / max(float(x.norm()), eps)
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            p = x @ x.T
            x = a * x + (b * p + c * p @ p) @ x
        else:
            p = x.T @ x
            x = a * x + x @ (b * p + c * p @ p)
    return x


def check(got, ref, rel, what):
    """Relative L2 error at most rel, and no element off by more than rel of itself plus 6 rel of the array's RMS."""
    got = torch.as_tensor(got).double().cpu().numpy()
    ref = torch.as_tensor(ref).double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.size == 0:
        return
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    rms = math.sqrt((ref ** 2).mean())
    l2 = math.sqrt((err ** 2).mean())
    assert l2 <= rel * rms + 1e-30, (what, l2 / max(rms, 1e-300), rel)
    worst = (err - rel * np.abs(ref)).max()
    assert worst <= 6 * rel * rms + 1e-30, (what, worst / max(rms, 1e-300), rel)
