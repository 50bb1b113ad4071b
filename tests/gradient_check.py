"""Gradients of the gated feed-forward block against differences of its loss.

A difference along a random direction says little: for a gradient of n elements
the slope is 1 / sqrt(n) of the norms' product, and so small against any
tolerance in the norms that a gradient of zeros passes.  Here each direction is
a part of the gradient under test (all of it, single rows, single columns),
scaled to length one: the slope along it has to be the part's own norm."""
import math

import torch

D = torch.float64


def gate(g, silu):
    """The activation by its definition."""
    if silu:
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def block_loss(x, w, dh, silu):
    """sum dh h: its gradients are dx and dw."""
    inter = w.shape[0] // 2
    gu = x @ w.T
    return (dh * gate(gu[:, :inter], silu) * gu[:, inter:]).sum()


def parts(t):
    """Masks: everything, and a few rows and columns."""
    yield "all", torch.ones_like(t)
    for axis in (0, 1):
        for at in sorted({0, t.shape[axis] // 2, t.shape[axis] - 1}):
            mask = torch.zeros_like(t)
            mask.select(axis, at).fill_(1)
            yield f"{('row', 'column')[axis]} {at}", mask


def check_block_gradients(x, w, dh, silu, dx, dw, rel):
    """dx and dw (float64) are within `rel` of every part's norm."""
    eps, floor = 1e-5, 1e-6   # differences: eps^2 of third derivatives, 2^-52 of the loss over eps
    for name, at, grad, loss in (("dx", x, dx, lambda t: block_loss(t, w, dh, silu)), ("dw", w, dw, lambda t: block_loss(x, t, dh, silu))):
        for part, mask in parts(grad):
            v = grad * mask
            norm = v.norm()
            assert norm > 0, f"{name}, {part}: no gradient"
            v = v / norm
            slope = (loss(at + eps * v) - loss(at - eps * v)) / (2 * eps)
            assert abs(slope - norm) <= rel * norm + floor, f"{name}, {part}: {norm.item()} against a slope of {slope.item()}"
