"""The float64 definition that the attention is checked against: equal to the recurrence row by row, its gradients to
differences (no GPU needed)."""
import pytest
import torch

import attention_oracle as ao


def inputs(rows, H, K, dk, dv, n_seq, per_row, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return (r(rows, H, dk), r(rows, K, dk), r(rows, K, dv), r(rows, K) if per_row else r(K)), r(n_seq, K, dk, dv), r


@pytest.mark.parametrize("per_row", [True, False])
def test_pairs_equal_the_recurrence(per_row):
    off = [0, 5, 5, 17, 18]
    x, state, _ = inputs(18, 6, 2, 3, 4, 4, per_row)
    got = ao.attention(*x, off, state, 0.7)
    y, last = ao.recurrence(*x, off, state, 0.7)
    assert torch.allclose(got["y"], y, rtol=1e-12, atol=1e-12)
    assert torch.allclose(got["last"], last, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("per_row", [True, False])
def test_gradients_equal_differences(per_row):
    """Central differences with a step of 1e-5: truncation and rounding below 1e-8 of the values."""
    off = [0, 4, 4, 11]
    x, state, r = inputs(11, 4, 2, 3, 2, 3, per_row, seed=1)
    dy, d_last = r(11, 4, 2), r(3, 2, 3, 2)
    got = ao.attention(*x, off, state, 0.5, dy, d_last)
    at = dict(zip(("q", "k", "v", "gate", "state"), (*x, state)))

    def loss(**new):
        t = {**at, **new}
        o = ao.recurrence(t["q"], t["k"], t["v"], t["gate"], off, t["state"], 0.5)
        return (o[0] * dy).sum() + (o[1] * d_last).sum()

    for name, t in at.items():
        d = r(*t.shape)
        slope = (loss(**{name: t + 1e-5 * d}) - loss(**{name: t - 1e-5 * d})) / 2e-5
        assert abs(slope - (got[name] * d).sum()) <= 1e-6 * (1 + abs(slope)), name
