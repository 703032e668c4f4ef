"""Train a scene's appearance: a feature table that primitives share, and a shading network.

One step reads every primitive's features from the table, drops some of them, renders them to a
feature image, shades it by a small channels-last network (a dense layer, the normalisation, a
hidden layer with dropout around which its input is passed, the colours) and compares the
colours with a target; the gradients run back through all of it, and the network's matrices
move by orthogonalised momentum.

    python examples/train_appearance.py --steps 50 --dropout 0.1

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


def shade(img, w1, gain, bias, wh, bh, w2, bias2, dropout=0.0, rng=None):
    """Colours [..., 3] of a feature image [1, pixels, channels]."""
    h = A.linear(img, w1)
    h = A.group_norm(h, GROUPS, gain, bias, act="silu")
    h = A.linear(h, wh, bh, act="silu", residual=h, p=dropout, rng=rng)
    return A.linear(h, w2, bias2)


def train(steps=50, n=30_000, width=320, height=192, lr=0.02, seed=0, device="cuda:0", log=None, dropout=0.0):
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
    wh = parameter(HIDDEN, HIDDEN, scale=0.1 * HIDDEN ** -0.5)
    gain = torch.ones(HIDDEN, device=device, requires_grad=True)
    bias, bh, bias2 = (torch.zeros(k, device=device, requires_grad=True) for k in (HIDDEN, HIDDEN, 3))
    matrices, others = [w1, wh, w2], [table, gain, bias, bh, bias2]
    momentum = [torch.zeros_like(m) for m in matrices]
    adam = torch.optim.Adam(others, lr=lr)
    losses = []
    for step in range(steps):
        feat = A.lookup(table, ids, scale=CHANNELS ** -0.5)
        if dropout > 0.0:                                            # an offset of its own beside the hidden layer's
            feat = A.dropout(feat, dropout, (seed, steps + step))
        img = render(rz, feat=feat)                                  # [channels][height][width], flat
        img = rz.view_images(img)[0].permute(1, 2, 0)                # channels last
        rgb = shade(img.reshape(1, height * width, CHANNELS), w1, gain, bias, wh, bh, w2, bias2, dropout, (seed, step))
        rgb = rgb.view(height, width, 3)
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
    ap.add_argument("--dropout", type=float, default=0.0, help="probability in the features and in the hidden layer")
    a = ap.parse_args()
    train(a.steps, n=a.primitives, dropout=a.dropout, log=lambda s: print(s, flush=True))
