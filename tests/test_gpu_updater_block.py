"""A block of the updater, trained: norm, projection, linear attention, norm with the residual, feed-forward, AdamW.

    n = norm(x),  q | k | v | gate = project(n),  z, h = norm(attention(q, k, v, gate), x),  out = ffn(z),  L = <out, c> + <h, e>

Tolerance in float32 (relative L2), u = 2^-24: every one of the ten passes, five forward and five backward, is within
(16 + 2 sqrt(K)) u of its formula with K = 700 rows the longest sum, 69 u; errors are carried on through Jacobians that are
at most 4 times as large for an error as for the values themselves: 10 x 69 x 4 u = 1.7e-4.
"""
import pytest
import torch

import attention_oracle as ao
import updater_oracle as o

pytestmark = pytest.mark.gpu
D, H, K, DK, DV, HIDDEN, EPS = 72, 6, 3, 20, 12, 136, 1e-6
WIDTHS = (H * DK, K * DK, K * DV, K)
TOLERANCE = 1.7e-4
NAMES = ("norm1", "gate1", "up1", "down1", "norm2", "gate2", "up2", "down2")
assert H * DV == D  # the attention's output is added to the stream


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def weights(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5

    return {"norm1": 1 + 0.1 * r(D), "gate1": r(HIDDEN, D), "up1": r(HIDDEN, D), "down1": 2 * r(sum(WIDTHS), HIDDEN),
            "norm2": 1 + 0.1 * r(D), "gate2": r(HIDDEN, D), "up2": r(HIDDEN, D), "down2": r(D, HIDDEN)}


def data(rows, n_seq, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*s, generator=g, device="cuda") for s in ((rows, D), (rows, D), (rows, D), (n_seq, K, DK, DV))]


class Block:
    """The operators over weights w of one type (the norms' in float32); the stream is float32."""

    def __init__(self, w, dtype):
        m = gsr()
        self.dtype = dtype
        self.norm1, self.norm2 = m.ResidualNorm(w["norm1"], dtype, EPS), m.ResidualNorm(w["norm2"], dtype, EPS)
        self.project = m.GatedFFN(w["gate1"], w["up1"], w["down1"])
        self.ffn = m.GatedFFN(w["gate2"], w["up2"], w["down2"])
        self.attention = m.LinearAttention(H, DK, DV, dtype, kv_heads=K)

    def split(self, p):
        q, k, v, gate = p.split(WIDTHS, dim=1)
        return q.unflatten(1, (H, DK)), k.unflatten(1, (K, DK)), v.unflatten(1, (K, DV)), gate

    def forward(self, x, state, offsets, last=None):
        """One pass, e.g. of single tokens with their states changed in place."""
        n, h = self.norm1.forward(x.to(self.dtype), h=torch.empty_like(x))
        y, last = self.attention.forward(*self.split(self.project.forward(n)), state=state, offsets=offsets, last=last)
        z, h = self.norm2.forward(y.flatten(1), residual=h)
        return self.ffn.forward(z), h, last

    def train(self, x, c, e, state, offsets):
        n, h0 = self.norm1.forward(x.to(self.dtype), h=torch.empty_like(x))
        p, saved1 = self.project.forward(n, save=True)
        parts = self.split(p)
        y, last, saved = self.attention.forward(*parts, state=state, offsets=offsets, save=True)
        z, h = self.norm2.forward(y.flatten(1), residual=h0)
        out, saved2 = self.ffn.forward(z, save=True)
        g2 = self.ffn.backward(z, saved2, c.to(self.dtype))
        b2 = self.norm2.backward(h, g2["x"], dh=e)
        dp = torch.empty_like(p)
        into = dict(zip(("q", "k", "v", "gate"), self.split(dp)))
        into["state"] = torch.empty_like(state)
        self.attention.backward(*parts, saved, b2["x"].unflatten(1, (H, DV)), state=state, offsets=offsets, grads=into)
        g1 = self.project.backward(n, saved1, dp)
        b1 = self.norm1.backward(h0, g1["x"], dh=b2["residual"])
        return (out, h, last), {"x": b1["residual"], "state": into["state"], "norm1": b1["weight"], "norm2": b2["weight"],
                                "gate1": g1["w_gate"], "up1": g1["w_up"], "down1": g1["w_down"],
                                "gate2": g2["w_gate"], "up2": g2["w_up"], "down2": g2["w_down"]}


def reference(w, x, c, e, state, offsets):
    leaf = {k: v.double().requires_grad_() for k, v in (*w.items(), ("x", x), ("state", state))}

    def norm(h, weight):
        return h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * weight

    def ffn(v, k):
        return (torch.nn.functional.silu(v @ leaf["gate" + k].T) * (v @ leaf["up" + k].T)) @ leaf["down" + k].T

    p = ffn(norm(leaf["x"], leaf["norm1"]), "1")
    q, k, v, gate = p.split(WIDTHS, dim=1)
    ys, lasts = [], []
    for s in range(len(offsets) - 1):
        a, b = offsets[s], offsets[s + 1]
        y, S = ao.sequence(q[a:b].unflatten(1, (H, DK)), k[a:b].unflatten(1, (K, DK)), v[a:b].unflatten(1, (K, DV)), gate[a:b],
                           leaf["state"][s], DK ** -0.5)
        ys.append(y)
        lasts.append(S)
    h = leaf["x"] + torch.cat(ys).flatten(1)
    out = ffn(norm(h, leaf["norm2"]), "2")
    loss = (out * c.double()).sum() + (h * e.double()).sum()
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    return (out.detach(), h.detach(), torch.stack(lasts).detach()), grads


OFFSETS = [0, 1, 1, 130, 600, 700]


def test_block_against_float64():
    w = weights()
    x, c, e, state = data(OFFSETS[-1], len(OFFSETS) - 1)
    got, grads = Block(w, torch.float32).train(x, c, e, state, torch.tensor(OFFSETS, device="cuda"))
    want, wgrads = reference(w, x, c, e, state, OFFSETS)
    for name, a, b in zip(("out", "h", "last"), got, want):
        assert (a.double() - b).norm() <= TOLERANCE * b.norm(), name
    for name in wgrads:
        assert (grads[name].double() - wgrads[name]).norm() <= TOLERANCE * wgrads[name].norm(), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
def test_single_tokens_go_on_with_a_sequence(dtype):
    """Four sequences of 33 rows at once, and the same row by row with the states carried.  16 bits: five operators, each
    rounding its output, by Jacobians of up to 4: 20 u."""
    w = {k: v if k.startswith("norm") else v.to(dtype) for k, v in weights().items()}
    x, _, _, state = data(4 * 33, 4, seed=2)
    block = Block(w, dtype)
    out, _, last = block.forward(x, state, None)
    carried, rows = state.clone(), x.view(4, 33, D)
    steps = [block.forward(rows[:, t].contiguous(), carried, None, last=carried)[0] for t in range(33)]
    tol = TOLERANCE if dtype == torch.float32 else 20 * o.UNIT[dtype]
    got = torch.stack(steps, 1).reshape(4 * 33, D).double()
    assert (got - out.double()).norm() <= tol * out.double().norm()
    assert (carried - last).norm() <= tol * last.norm()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training(bits):
    """Forward, backward and AdamW with 16-bit copies in one graph, replayed between the program's own work: every replay
    gives the bits of the eager step."""
    rows, offsets = 700, torch.tensor(OFFSETS, device="cuda")

    def setup():
        master = weights(3)
        low = {k: v if k.startswith("norm") else v.bfloat16() for k, v in master.items()}
        opt = gsr().AdamW([master[k] for k in NAMES], lr=0.01, weight_decay=0.01, state_bits=bits,
                          copies=[None if k.startswith("norm") else low[k] for k in NAMES])
        return master, Block(low, torch.bfloat16), opt

    x, c, e, state = data(rows, len(OFFSETS) - 1, seed=4)
    eager, block, opt = setup()
    captured, block2, opt2 = setup()
    _, warm = block2.train(x, c, e, state, offsets)  # loads the kernels; changes no weight
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out2, _, _), grads2 = block2.train(x, c, e, state, offsets)
        opt2.step([grads2[k] for k in NAMES])
    assert int(opt2.steps) == 0
    for k in range(4):
        for t, n in zip((x, c, e, state), data(rows, len(OFFSETS) - 1, seed=5 + k)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        (out, _, _), grads = block.train(x, c, e, state, offsets)
        opt.step([grads[n] for n in NAMES])
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and int(opt.steps) == int(opt2.steps) == k + 1
        for n in NAMES:
            assert torch.equal(grads[n], grads2[n]) and torch.equal(eager[n], captured[n]), n
