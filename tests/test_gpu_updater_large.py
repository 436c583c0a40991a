"""The norm, the optimizer and the attention on arrays whose offsets pass 32 bits, and on shared scratch memory: what lies
far out is compared with the same rows by themselves, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 2 ** 20


def gsr():
    import gaussian_splatting_rasterizer_amd as m
    return m


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


@pytest.fixture
def gen():
    yield torch.Generator(device="cuda").manual_seed(0)
    torch.cuda.empty_cache()


def test_norm_of_many_values(gen):
    """Rows spread over 2^31 + 2^20 values, and as many rows as fill them."""
    width, dtype = 512, torch.bfloat16
    w = randn(gen, width)
    norm = gsr().ResidualNorm(w, dtype)
    rows = FAR // width
    x = torch.zeros(rows, width, dtype=dtype, device="cuda")
    x[-5:] = randn(gen, 5, width, dtype=dtype)
    x[0] = 1
    few = x[-5:].clone()
    y, _ = norm.forward(x)
    want, _ = norm.forward(few)
    assert torch.equal(y[-5:], want)
    assert (y[1:-5] == 0).all()  # of either sign
    codes, scales, _ = norm.forward8(x, group=128)
    c5, s5, _ = norm.forward8(few, group=128)
    assert torch.equal(codes[-5:].view(torch.uint8), c5.view(torch.uint8)) and torch.equal(scales[-5:], s5)
    del codes, scales
    g, g5 = norm.backward(x, y)["x"], norm.backward(few, want)["x"]
    assert torch.equal(g[-5:], g5)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_of_many_values(gen, bits):
    p, g = (torch.zeros(FAR + 100, device="cuda") for _ in range(2))
    p[-700:], g[-700:] = randn(gen, 700), randn(gen, 700)
    first = FAR + 100 - (FAR + 100) % 256 - 512  # a block's first value
    p2, g2 = p[first:].clone(), g[first:].clone()
    opt, few = gsr().AdamW([p], lr=0.1, state_bits=bits), gsr().AdamW([p2], lr=0.1, state_bits=bits)
    for _ in range(2):
        opt.step([g])
        few.step([g2])
    assert torch.equal(p[first:], p2)
    assert torch.equal(opt.v[0][first:].view(torch.uint8), few.v[0].view(torch.uint8))
    assert (p[:first - 512] == 0).all()


def test_attention_of_heads_far_apart(gen):
    """Heads 2^31 values apart, in inputs, outputs and gradients."""
    rows, K, d, dtype = 700, 2, 64, torch.bfloat16
    far = torch.empty(FAR + 4 * rows * d, dtype=dtype, device="cuda")
    k = torch.as_strided(far, (rows, K, d), (d, FAR, 1))
    v = torch.as_strided(far, (rows, K, d), (d, FAR, 1), rows * d)
    y, dk = (torch.as_strided(far, (rows, K, d), (d, FAR, 1), i * rows * d) for i in (2, 3))
    k2, v2 = randn(gen, rows, K, d, dtype=dtype) * 0.1, randn(gen, rows, K, d, dtype=dtype)
    k.copy_(k2)
    v.copy_(v2)
    q, gate, dy = randn(gen, rows, K, d, dtype=dtype), randn(gen, rows, K) + 3, randn(gen, rows, K, d, dtype=dtype)
    att = gsr().LinearAttention(K, d, d, dtype)
    _, last, saved = att.forward(q, k, v, gate, y=y, save=True)
    y2, last2, saved2 = att.forward(q, k2, v2, gate, save=True)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    got = att.backward(q, k, v, gate, saved, dy, grads={"k": dk, "gate": torch.empty_like(gate)})
    want = att.backward(q, k2, v2, gate, saved2, dy)
    assert torch.equal(dk, want["k"]) and torch.equal(got["gate"], want["gate"])


def test_attention_of_states_beyond_32_bits(gen):
    """70000 states of 2 x 128 x 128: 2^31 values and more; the last ones against themselves, in place."""
    n, K, d, dtype = 70000, 2, 128, torch.bfloat16
    q, k, v = (randn(gen, n, K, d, dtype=dtype) for _ in range(3))
    gate = randn(gen, n, K)
    state = torch.zeros(n, K, d, d, device="cuda")
    assert state.numel() > 2 ** 31
    state[-3:] = randn(gen, 3, K, d, d)
    few = state[-3:].clone()
    att = gsr().LinearAttention(K, d, d, dtype)
    y, _ = att.forward(q, k, v, gate, state=state, last=state)
    y2, last = att.forward(q[-3:], k[-3:], v[-3:], gate[-3:], state=few)
    assert torch.equal(y[-3:], y2) and torch.equal(state[-3:], last)


def test_captured_attention_among_larger_calls(gen):
    """The graph goes on using the scratch memory it was captured with while the object's grows, and smaller calls between
    the replays use what the object holds then."""
    dtype, K, d = torch.bfloat16, 2, 64
    att = gsr().LinearAttention(K, d, d, dtype)

    def call(t):
        y, last, saved = att.forward(*t[:4], save=True)
        return y, last, att.backward(*t[:4], saved, t[4])

    def inputs(rows):
        return [randn(gen, rows, K, d, dtype=dtype), randn(gen, rows, K, d, dtype=dtype) * 0.1,
                randn(gen, rows, K, d, dtype=dtype), randn(gen, rows, K) + 3, randn(gen, rows, K, d, dtype=dtype)]

    t = inputs(1500)
    call(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last, grads = call(t)
    for rows in (40000, 90000, 600):
        for a, b in zip(t, inputs(1500)):
            a.copy_(b)
        call(inputs(rows))
        graph.replay()
        other = call(inputs(rows))
        y2, last2, grads2 = call(t)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(last, last2)
        assert all(torch.equal(grads[n], grads2[n]) for n in grads)
        del other


def test_two_objects_on_two_streams(gen):
    dtype, K, d, rows = torch.float16, 2, 64, 20000
    t = [[randn(gen, rows, K, d, dtype=dtype) for _ in range(3)] + [randn(gen, rows, K) + 2] for _ in range(2)]
    want = [gsr().LinearAttention(K, d, d, dtype).forward(*x) for x in t]
    objects = [gsr().LinearAttention(K, d, d, dtype) for _ in t]
    streams = [torch.cuda.Stream() for _ in t]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [a.forward(*x, stream=s) for a, x, s in zip(objects, t, streams)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for (y, last), (y2, last2) in zip(got, want):
        assert torch.equal(y, y2) and torch.equal(last, last2)
