"""Train a scene's appearance: a feature table that primitives share, and a shading network.

One step reads every primitive's features from the table, renders them to a feature
image, shades it by a small channels-last network and compares the colours with a target;
the gradients run back through all of it, and the network's matrices move by
orthogonalised momentum.

    python examples/train_appearance.py --steps 50

The target is the same geometry with colours of its own, so the loss can fall far but not
to zero: 256 table entries stand for all primitives.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sphere_rasterization_amd import appearance as A
from sphere_rasterization_amd import scenes as S
from sphere_rasterization_amd.autograd import render
from sphere_rasterization_amd.raster import Rasterizer

CHANNELS, HIDDEN, GROUPS, ENTRIES = 16, 32, 8, 256


def target_image(scene, palette, ids, device):
    """Colours of the entries, rendered: what the trained table and network should show."""
    own = S.driving(n=scene.n, width=scene.cams[0].width, height=scene.cams[0].height, channels=3)
    own.feat = np.ascontiguousarray(palette[ids], np.float32)
    rz = Rasterizer(own, device=device)
    rz.forward()
    return rz.view_images()[0].permute(1, 2, 0).contiguous()


def train(steps=50, n=30_000, width=320, height=192, lr=0.02, seed=0, device="cuda:0", log=None):
    """Loss of each step."""
    rng = np.random.default_rng(seed)
    torch.manual_seed(seed)
    scene = S.driving(n=n, width=width, height=height, channels=CHANNELS)
    ids_np = rng.integers(0, ENTRIES, n)
    target = target_image(scene, rng.uniform(0.0, 1.0, (ENTRIES, 3)), ids_np, device)
    ids = torch.from_numpy(ids_np).to(device)
    rz = Rasterizer(scene, device=device)

    def parameter(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device=device)).requires_grad_()

    table = parameter(ENTRIES, CHANNELS, scale=0.5)
    w1, w2 = parameter(CHANNELS, HIDDEN, scale=CHANNELS ** -0.5), parameter(HIDDEN, 3, scale=0.1)
    gain = torch.ones(HIDDEN, device=device, requires_grad=True)
    bias, bias2 = torch.zeros(HIDDEN, device=device, requires_grad=True), torch.zeros(3, device=device, requires_grad=True)
    matrices, others = [w1, w2], [table, gain, bias, bias2]
    momentum = [torch.zeros_like(m) for m in matrices]
    adam = torch.optim.Adam(others, lr=lr)
    losses = []
    for step in range(steps):
        feat = A.lookup(table, ids, scale=CHANNELS ** -0.5)
        img = render(rz, feat=feat)                                  # [channels][height][width], flat
        h = rz.view_images(img)[0].permute(1, 2, 0)[None]            # channels last
        h = A.group_norm(h.reshape(1, height * width, CHANNELS) @ w1, GROUPS, gain, bias, act="silu")
        rgb = (h @ w2 + bias2).view(height, width, 3)
        loss = (rgb - target).square().mean()
        adam.zero_grad()
        for m in matrices:
            m.grad = None
        loss.backward()
        adam.step()
        with torch.no_grad():
            for m, v in zip(matrices, momentum):
                v.mul_(0.9).add_(m.grad, alpha=0.1)
                # a step of the same size for every direction, whatever the matrix's shape
                m.add_(A.orthogonalize(v, scale=max(1.0, m.shape[0] / m.shape[1]) ** 0.5), alpha=-lr)
        losses.append(float(loss.detach()))
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--primitives", type=int, default=30_000)
    a = ap.parse_args()
    train(a.steps, n=a.primitives, log=lambda s: print(s, flush=True))
