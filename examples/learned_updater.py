"""A learned recurrent updater on top of the renderer, trained end to end.

    python examples/learned_updater.py [--gaussians 20000] [--updates 4] [--steps 40] [--dtype bfloat16]

Each update renders the scene, replays the scores and turns every Gaussian's token into a change of its parameters
("Final Token and Updater" of the Renderer Score Tokens proposal: a projection of the token, a hidden state per
Gaussian, a parameter update):

    p = block(token),  h <- sigma(p_gate) h + (1 - sigma(p_gate)) p_x,  delta = readout(h),  theta <- theta + delta

The roll-out uses the operators one row per Gaussian and keeps only the states.  Training then runs each operator once
over all updates (the recurrence over one sequence per Gaussian), with dL/d(delta) from the renderer's backward pass,
and takes an orthogonalised momentum step on every weight.  Tokens are inputs: no gradient flows into them.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gaussian_splatting_rasterizer_amd as gsr  # noqa: E402
import scenes  # noqa: E402


class Updater:
    """Token block, recurrence and readout; float32 master weights and momenta, operands in `dtype`."""

    def __init__(self, token_width, n_params, channels=64, hidden=256, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        shapes = {"gate1": (hidden, token_width), "up1": (hidden, token_width), "down1": (2 * channels, hidden),
                  "gate2": (hidden, channels), "up2": (hidden, channels), "down2": (n_params, hidden)}
        self.master = {k: torch.randn(s, generator=gen, device=device) * s[1] ** -0.5 for k, s in shapes.items()}
        self.master["down2"].zero_()  # the first update changes nothing
        self.momentum = {k: torch.zeros_like(w) for k, w in self.master.items()}
        w = self.weights = {k: v.to(dtype, copy=True) for k, v in self.master.items()}
        self.dtype, self.channels = dtype, channels
        self.block = gsr.GatedFFN(w["gate1"], w["up1"], w["down1"], activation="gelu")
        self.scan = gsr.GatedScan(channels, dtype, device=device)
        self.readout = gsr.GatedFFN(w["gate2"], w["up2"], w["down2"], activation="silu")
        self.ortho = {s: gsr.Orthogonalizer(1, *s, torch.float32, device=device) for s in set(shapes.values())}

    def update(self, tokens, state):
        """One update: tokens [n, token_width] and the states [n, channels] (changed in place) -> delta [n, n_params]."""
        p = self.block.forward(tokens)
        c = self.channels
        y, _ = self.scan.forward(p[:, :c], p[:, c:], h0=state, h_last=state)
        return self.readout.forward(y)

    def gradients(self, tokens, d_delta, n):
        """Weight gradients for tokens [n * updates, token_width] (a Gaussian's updates in a row) and dL/d(delta)."""
        c = self.channels
        p, saved_block = self.block.forward(tokens, save=True)
        h0 = torch.zeros((n, c), device=tokens.device)
        y, _, saved_scan = self.scan.forward(p[:, :c], p[:, c:], h0=h0, save=True)
        _, saved_readout = self.readout.forward(y, save=True)
        g2 = self.readout.backward(y, saved_readout, d_delta)
        dp = torch.empty_like(p)
        self.scan.backward(p[:, :c], p[:, c:], saved_scan, g2["x"], h0=h0, grads={"gate": dp[:, :c], "x": dp[:, c:]})
        grads = self.block.new_grads(tokens.shape[0])
        del grads["x"]
        g1 = self.block.backward(tokens, saved_block, dp, grads=grads)
        return {"gate1": g1["w_gate"], "up1": g1["w_up"], "down1": g1["w_down"],
                "gate2": g2["w_gate"], "up2": g2["w_up"], "down2": g2["w_down"]}

    def step(self, grads, lr, momentum=0.9):
        for k, w in self.master.items():
            m = self.momentum[k].mul_(momentum).add_(grads[k].float())
            o = self.ortho[tuple(w.shape)].run(m)
            w.add_(o, alpha=-lr * math.sqrt(max(1.0, w.shape[0] / w.shape[1])))
            self.weights[k].copy_(w)


class Fit:
    """A scene whose parameters are to be moved so that its render matches `observed` [V, H, W, 3]."""

    def __init__(self, scene, observed, dtype):
        self.r = gsr.rasterizer_for_scene(scene)
        self.observed, self.dtype = observed, dtype
        r = self.r
        self.start = torch.cat([r.means, r.quats, r.scales.log(), torch.logit(r.opacities, eps=1e-6)[:, None],
                                r.sh.reshape(r.n, -1)], dim=1)
        self.n, self.token_width = self.r.n, 9 + 3 * self.r.d
        self.n_params = 11 + 3 * self.r.d
        sizes = (3, 4, 3, 1, 3 * self.r.d)
        reach = (0.01, 0.01, 0.02, 0.05, 0.02)  # size of a unit of delta, per parameter group
        self.scale = torch.cat([torch.full((s,), v) for s, v in zip(sizes, reach)]).to(self.r.device)
        self.outputs, self.grads = self.r.new_outputs(), self.r.new_grads()

    def reset(self):
        self.theta = self.start.clone()
        self.apply(0.0)

    def apply(self, delta):
        r, t = self.r, self.theta
        t += delta * self.scale
        r.means.copy_(t[:, :3])
        r.quats.copy_(t[:, 3:7])
        r.scales.copy_(t[:, 7:10].exp())
        r.opacities.copy_(t[:, 10].sigmoid())
        r.sh.copy_(t[:, 11:].reshape(r.sh.shape))

    def render(self):
        """-> the loss, half the squared error summed over the images, and the residual."""
        self.r.project_and_bin()
        color, _, _ = self.r.render(self.outputs)
        residual = color - self.observed
        return 0.5 * (residual.double() ** 2).sum(), residual

    def tokens(self):
        """Score tokens of the current render, compressed to (-1, 1) by their column's RMS."""
        t = self.r.score_replay(self.observed)
        rms = t.pow(2).mean(dim=0, keepdim=True).sqrt() + 1e-12
        return (t / (t.abs() + rms)).to(self.dtype)

    def parameter_gradient(self, residual):
        """dL/d(delta) of a change made just before the last render, [n, n_params]."""
        r, g = self.r, self.r.backward(residual, self.grads)
        o = r.opacities
        raw = torch.cat([g["means"], g["quats"], g["scales"] * r.scales, (g["opacities"] * o * (1 - o))[:, None],
                         g["sh"].reshape(self.n, -1)], dim=1)
        return raw * self.scale


def roll_out(fit, updater, updates, train=True):
    """Runs `updates` updates from the start.  -> losses (after 0, 1, ... updates), and for training the tokens
    [n * updates, ...] and dL/d(delta) for the sum of the losses after each update."""
    fit.reset()
    state = torch.zeros((fit.n, updater.channels), device=fit.r.device)
    tokens = torch.empty((fit.n, updates, fit.token_width), dtype=fit.dtype, device=fit.r.device)
    grads = torch.zeros((fit.n, updates, fit.n_params), device=fit.r.device)
    loss, _ = fit.render()
    losses = [loss]
    for k in range(updates):
        tokens[:, k] = fit.tokens()
        fit.apply(updater.update(tokens[:, k], state))
        loss, residual = fit.render()
        losses.append(loss)
        if train:  # a change lasts: it counts for every later render
            grads[:, :k + 1] += fit.parameter_gradient(residual)[:, None]
    losses = torch.stack(losses)
    if not train:
        return losses
    # the step depends on the gradients' directions only, so they are scaled into the range of every type
    grads /= grads.abs().max().clamp_min(1e-30)
    return losses, tokens.reshape(-1, fit.token_width), grads.reshape(-1, fit.n_params).to(fit.dtype)


def train(scene, observed, updates=4, steps=40, lr=0.02, dtype=torch.bfloat16, report=None):
    """-> the losses of every roll-out, [steps + 1, updates + 1], and the updater."""
    fit = Fit(scene, observed, dtype)
    updater = Updater(fit.token_width, fit.n_params, dtype=dtype, device=fit.r.device)
    history = []
    for i in range(steps):
        losses, tokens, d_delta = roll_out(fit, updater, updates)
        updater.step(updater.gradients(tokens, d_delta, fit.n), lr)
        history.append(losses)
        if report:
            report(i, losses)
    history.append(roll_out(fit, updater, updates, train=False))
    return torch.stack(history), updater


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gaussians", type=int, default=20000)
    ap.add_argument("--updates", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--lr", type=float, default=0.02)
    ap.add_argument("--dtype", choices=("bfloat16", "float16", "float32"), default="bfloat16")
    a = ap.parse_args()
    scene = scenes.tiny_scene(n=a.gaussians, n_views=4, W=256, H=192, log_scale=(-4.0, 0.3))
    target = gsr.rasterizer_for_scene(scene.perturbed())
    target.project_and_bin()
    observed = target.render()[0]
    history, _ = train(scene, observed, a.updates, a.steps, a.lr, getattr(torch, a.dtype),
                       report=lambda i, l: print(f"step {i}: " + " ".join(f"{v:.2f}" for v in l.tolist()), flush=True))
    print("trained: " + " ".join(f"{v:.2f}" for v in history[-1].tolist()))


if __name__ == "__main__":
    main()
