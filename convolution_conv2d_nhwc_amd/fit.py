"""Fitting a head on the maps of a convolution layer, with the training-side
operators as they are used together:

    map  = conv(images)                    a frozen layer of conv_nhwc.h
    z    = group_norm(map), SiLU           statistics kept for the gradients
    loss = head_loss_grad(z, w, labels)    a class per pixel, gradients of z and w
    dgamma, dbeta from group_norm_grad     plain gradient steps
    w   -= rate * orthogonalize(momentum)  the head's update

``python -m convolution_conv2d_nhwc_amd.fit [--steps N]`` runs it on synthetic
images labelled by a fixed random head and prints the loss as it falls.
"""
from __future__ import annotations

import argparse
from typing import Optional

import torch

from . import _lib, train


class HeadFit:
    """A norm and a 1x1 head of `classes` on a layer's output map."""

    def __init__(self, layer: _lib.Conv2d, classes: int, groups: int = 8, rate: float = 0.1, momentum: float = 0.9,
                 seed: int = 0, device="cuda"):
        n, h, w, c = layer.out_shape
        g = torch.Generator(device=device).manual_seed(seed)
        self.layer, self.groups, self.rate, self.momentum = layer, groups, rate, momentum
        self.gamma = torch.ones(c, device=device)
        self.beta = torch.zeros(c, device=device)
        self.w = torch.randn((classes, c), generator=g, device=device) * (0.1 / c ** 0.5)
        self.velocity = torch.zeros_like(self.w)
        self.stats = torch.empty((n, groups, 2), device=device)
        # an orthogonal update of a tall matrix moves every class by less than that of a square one
        self.scale = max(1.0, classes / c) ** 0.5

    def features(self, images, weight, bias):
        """(map, normalised map) of the images under the frozen layer."""
        y = self.layer.run(images, weight, bias)
        z = train.group_norm(y, self.groups, self.gamma, self.beta, act="silu", stats=self.stats)
        return y, z

    def step(self, images, weight, bias, labels, pixel_weights: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One update; returns the loss before it (on the device)."""
        y, z = self.features(images, weight, bias)
        total, _, dz, dw = train.head_loss_grad(z, self.w.bfloat16(), labels, pixel_weights)
        _, dgamma, dbeta = train.group_norm_grad(dz, y, self.stats, self.gamma, self.beta, act="silu")
        self.velocity.mul_(self.momentum).add_(dw)
        self.w.add_(train.orthogonalize(self.velocity), alpha=-self.rate * self.scale)
        self.gamma.add_(dgamma, alpha=-self.rate)
        self.beta.add_(dbeta, alpha=-self.rate)
        return total

    def loss(self, images, weight, bias, labels) -> torch.Tensor:
        _, z = self.features(images, weight, bias)
        return train.head_loss(z, self.w.bfloat16(), labels)[0]


def synthetic(layer: _lib.Conv2d, classes: int, seed: int = 1, device="cuda"):
    """Images, the frozen layer's weights and a label per output pixel: the
    class that a fixed random head scores highest on the normalised map; a
    tenth of the pixels carry no label."""
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=device)

    c = layer.out_shape[3]
    images = randn(*layer.in_shape).bfloat16()
    weight = (randn(*layer.w_shape) * (2.0 / (layer.w_shape[1] * layer.w_shape[2] * layer.w_shape[3])) ** 0.5).bfloat16()
    bias = 0.1 * randn(c)
    z = train.group_norm(layer.run(images, weight, bias), 8, act="silu")
    teacher = (randn(classes, c) / c ** 0.5).bfloat16()
    labels = torch.matmul(z.float(), teacher.float().t()).argmax(-1)
    labels[torch.rand(labels.shape, generator=g, device=device) < 0.1] = -100
    return images, weight, bias, labels


def run(steps: int = 60, classes: int = 200, quiet: bool = False):
    """The losses of `steps` updates on a batch of 8 maps of 40x40x64."""
    layer = _lib.Conv2d(8, 40, 40, 32, 64, 3, 3, (1, 1), (1, 1), dtype="bf16")
    data = synthetic(layer, classes)
    fit = HeadFit(layer, classes)
    losses = [fit.step(*data) for _ in range(steps)]
    losses.append(fit.loss(*data))
    losses = [float(v) for v in torch.stack(losses).cpu()]
    if not quiet:
        for i in range(0, steps + 1, max(1, steps // 10)):
            print("step %4d  loss %.4f" % (i, losses[i]), flush=True)
    layer.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--classes", type=int, default=200)
    a = ap.parse_args()
    run(a.steps, a.classes)
