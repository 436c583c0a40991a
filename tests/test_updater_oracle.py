"""The float64 definitions of the updater's operators against differences and against what they must give."""
import numpy as np
import pytest
import torch

import updater_oracle as o

NS = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_ffn_gradient_against_differences(name):
    torch.manual_seed(0)
    t = {"x": torch.randn(5, 7).double(), "w_gate": torch.randn(6, 7).double(), "w_up": torch.randn(6, 7).double(),
         "w_down": torch.randn(4, 6).double()}
    dy = torch.randn(5, 4).double()
    ref = o.ffn(*t.values(), name, dy)
    eps = 1e-5
    for k in t:
        v = torch.randn(t[k].shape).double()
        hi, lo = dict(t), dict(t)
        hi[k], lo[k] = t[k] + eps * v, t[k] - eps * v
        diff = ((o.ffn(*hi.values(), name) - o.ffn(*lo.values(), name)) * dy).sum() / (2 * eps)
        got = (ref[k] * v).sum()
        assert abs(diff - got) <= 1e-8 * max(1.0, abs(got)), k


def test_scan_gradient_against_differences():
    rng = np.random.default_rng(1)
    off = [0, 3, 3, 9, 10]
    t = {"gate": rng.normal(size=(10, 3)), "x": rng.normal(size=(10, 3)), "h0": rng.normal(size=(4, 3))}
    dy, dl = rng.normal(size=(10, 3)), rng.normal(size=(4, 3))
    ref = o.scan(t["gate"], t["x"], off, t["h0"], dy, dl)
    eps = 1e-5

    def loss(q):
        r = o.scan(q["gate"], q["x"], off, q["h0"])
        return (r["y"] * dy).sum() + (r["h_last"] * dl).sum()

    for k in t:
        v = rng.normal(size=t[k].shape)
        hi, lo = dict(t), dict(t)
        hi[k], lo[k] = t[k] + eps * v, t[k] - eps * v
        diff = (loss(hi) - loss(lo)) / (2 * eps)
        assert abs(diff - (ref[k] * v).sum()) <= 1e-8, k
    assert np.array_equal(ref["h_last"][1], t["h0"][1]) and np.array_equal(ref["h0"][1], dl[1])  # the empty one


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (5, 5)])
def test_newton_schulz_acts_on_the_singular_values(shape):
    """The matrix polynomial maps each singular value s to a s + b s^3 + c s^5 and keeps the singular vectors."""
    torch.manual_seed(2)
    g = torch.randn(*shape).double()
    u, s, vt = torch.linalg.svd(g, full_matrices=False)
    s = s / g.norm()
    for _ in range(5):
        s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
    assert (o.newton_schulz(g, 5, NS) - u @ torch.diag(s) @ vt).abs().max() <= 1e-12
    assert s.max() < 1.25
