"""The example that trains an updater with all three operators and the renderer."""
import pytest
import torch

import scenes
import updater_oracle as o

pytestmark = pytest.mark.gpu


def setup(n=400):
    import gaussian_splatting_rasterizer_amd as gsr
    scene = scenes.tiny_scene(n=n, n_views=3, W=64, H=48, sh_degree=1)
    target = gsr.rasterizer_for_scene(scene.perturbed())
    target.project_and_bin()
    return scene, target.render()[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_training_lowers_the_loss(dtype):
    from examples import learned_updater as ex
    scene, observed = setup()
    history, _ = ex.train(scene, observed, updates=3, steps=25, dtype=dtype)
    h = history.cpu()
    assert torch.isfinite(h).all()
    assert (h[0] == h[0, 0]).all()       # the untrained readout is zero
    assert h[-1, -1] < 0.9 * h[-1, 0]    # the trained updates improve the scene
    assert h[-1, 1:].sum() < h[0, 1:].sum()


def test_weight_gradients_against_autograd():
    """float32, against float64 autograd of the definition over all updates.  Three operators in a row, forward and
    backward: 6 (16 + 2 sqrt(K)) u with K = 1200 rows the longest sum is 3e-5; 1e-4 leaves the Jacobians a factor 3."""
    from examples import learned_updater as ex
    scene, observed = setup()
    fit = ex.Fit(scene, observed, torch.float32)
    up = ex.Updater(fit.token_width, fit.n_params, dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    up.weights["down2"].copy_(torch.randn(up.weights["down2"].shape, generator=gen, device="cuda") * 0.05)
    updates, n = 3, fit.n
    _, tokens, d_delta = ex.roll_out(fit, up, updates)
    got = up.gradients(tokens, d_delta, n)

    w = {k: v.double().requires_grad_() for k, v in up.weights.items()}
    c = up.channels
    x = tokens.double()
    p = (torch.nn.functional.gelu(x @ w["gate1"].T) * (x @ w["up1"].T)) @ w["down1"].T
    p = p.reshape(n, updates, 2 * c)
    h, hs = torch.zeros(n, c, dtype=torch.float64, device="cuda"), []
    for k in range(updates):
        a = torch.sigmoid(p[:, k, :c])
        h = a * h + (1 - a) * p[:, k, c:]
        hs.append(h)
    y = torch.stack(hs, dim=1).reshape(-1, c)
    delta = (torch.nn.functional.silu(y @ w["gate2"].T) * (y @ w["up2"].T)) @ w["down2"].T
    (delta * d_delta.double()).sum().backward()
    for k, v in w.items():
        o.check(got[k], v.grad, 1e-4, k)


def test_roll_out_equals_one_pass():
    """One row per call with the states carried in place gives what one pass over each Gaussian's updates gives."""
    from examples import learned_updater as ex
    scene, observed = setup(n=150)
    fit = ex.Fit(scene, observed, torch.float32)
    up = ex.Updater(fit.token_width, fit.n_params, dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(2)
    tokens = torch.randn((150, 4, fit.token_width), generator=gen, device="cuda")
    state = torch.zeros((150, up.channels), device="cuda")
    for k in range(4):
        p = up.block.forward(tokens[:, k])
        y, _ = up.scan.forward(p[:, :up.channels], p[:, up.channels:], h0=state, h_last=state)
    p = up.block.forward(tokens.reshape(-1, fit.token_width))
    _, h = up.scan.forward(p[:, :up.channels], p[:, up.channels:], h0=torch.zeros_like(state))
    o.check(state, h, 16 * o.UNIT[torch.float32] * 8, "states")
