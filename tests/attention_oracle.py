"""Linear attention with a decay for each head from its definition in float64: every pair of rows of a sequence at once,
gradients by differentiation.  It uses nothing of the package."""
import math

import torch


def sequence(q, k, v, gate, S0, scale):
    """One sequence: q [T, H, dk], k [T, K, dk], v [T, K, dv], gate [T, K], S0 [K, dk, dv] -> y [T, H, dv], S_T."""
    T, H, K = q.shape[0], q.shape[1], k.shape[1]
    if T == 0:
        return q.new_zeros(0, H, v.shape[2]), S0
    c = torch.nn.functional.logsigmoid(gate).cumsum(0).t()  # [K, T]
    seen = torch.ones(T, T, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(seen, torch.exp(torch.where(seen, c[:, :, None] - c[:, None, :], 0.0)), 0.0)
    qh = q.transpose(0, 1).reshape(K, H // K, T, -1)
    kh, vh = k.transpose(0, 1)[:, None], v.transpose(0, 1)[:, None]
    weights = (qh @ kh.transpose(2, 3)) * decay[:, None]
    y = weights @ vh + torch.exp(c)[:, None, :, None] * (qh @ S0[:, None])
    S = torch.exp(c[:, -1])[:, None, None] * S0 + (kh[:, 0] * torch.exp(c[:, -1:] - c)[..., None]).transpose(1, 2) @ vh[:, 0]
    return scale * y.reshape(H, T, -1).transpose(0, 1), S


def attention(q, k, v, gate, offsets, state, scale, dy=None, d_last=None):
    """offsets: a list.  -> dict of y, last and, with dy, the gradients q, k, v, gate, state."""
    leaf = {n: t.detach().double().requires_grad_(dy is not None)
            for n, t in (("q", q), ("k", k), ("v", v), ("gate", gate), ("state", state))}
    rows = leaf["gate"] if gate.dim() == 2 else leaf["gate"][None].expand(q.shape[0], -1)
    ys, lasts, loss = [], [], 0.0
    for s in range(len(offsets) - 1):
        a, b = offsets[s], offsets[s + 1]
        y, S = sequence(leaf["q"][a:b], leaf["k"][a:b], leaf["v"][a:b], rows[a:b], leaf["state"][s], scale)
        ys.append(y)
        lasts.append(S)
        if dy is not None:
            loss = loss + (y * dy[a:b].double()).sum()
            if d_last is not None:
                loss = loss + (S * d_last[s].double()).sum()
    out = {"y": torch.cat(ys).detach(), "last": torch.stack(lasts).detach()}
    if dy is not None:
        names = list(leaf)
        got = torch.autograd.grad(loss, [leaf[n] for n in names], allow_unused=True)
        out.update({n: g if g is not None else torch.zeros_like(leaf[n]) for n, g in zip(names, got)})
    return out


def recurrence(q, k, v, gate, offsets, state, scale):
    """The same forward pass row by row, as the formula is written."""
    q, k, v, state = (t.double() for t in (q, k, v, state))
    a = torch.sigmoid(gate.double())
    G = q.shape[1] // k.shape[1]
    y, last = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64, device=q.device), state.clone()
    for s in range(len(offsets) - 1):
        S = state[s]
        for t in range(offsets[s], offsets[s + 1]):
            S = (a[t] if a.dim() == 2 else a)[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * torch.matmul(q[t].view(S.shape[0], G, -1), S).reshape(q.shape[1], -1)
        last[s] = S
    return y, last


V = 2.0 ** -24


def root(n):
    return math.sqrt(max(n, 1))
